"""The few-token layer where part of its grid never becomes resident: the workgroups that are there find the others'
gate/up chunks and do them, with the same arithmetic.

A test entry of the library (not in the header) launches fewer workgroups of the experts kernel than the chunks are
dealt to.  Every launched workgroup waits only for chunks that it or another launched one can take, so each call ends.
"""
import contextlib

import pytest
import torch

import sparse_moe_layer_amd as lib
import test_parity_few as tf

pytestmark = pytest.mark.gpu


@contextlib.contextmanager
def present(workgroups):
    lib.LIB.moe_test_few_present(workgroups)
    try:
        yield
    finally:
        lib.LIB.moe_test_few_present(0)


def same_bits(p, workgroups):
    ref, ids, w = tf.run_few(p)
    torch.cuda.synchronize()
    for n in workgroups:
        print(f"[absent] {p.cfg.name}: {n} workgroups there", flush=True)
        with present(n):
            out, i2, w2 = tf.run_few(p)
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), ref.view(torch.int16)), f"{n} workgroups: other bits"
        assert torch.equal(ids, i2) and torch.equal(w, w2)
    return ref, ids, w


@pytest.mark.parametrize("wdt", ["bf16", "fp8", "mxfp4"])
@pytest.mark.parametrize("T,H,E,k,I,Is", [
    (16, 256, 64, 8, 640, 64),    # more slabs than waves: a chunk is a wave's slab
    (1, 1024, 4, 4, 128, 0),      # few slabs: eight waves share one
    (3, 1024, 16, 4, 256, 128),   # some slabs: a chunk is a few of them, the last chunk short
    (5, 640, 33, 3, 384, 104),
])
def test_absent_workgroups_change_no_bit(T, H, E, k, I, Is, wdt):
    p = tf.few_problem(T, H, E, k, I, Is, wdt, seed=T)
    tf.check_few(p, *same_bits(p, (255, 128, 17, 1)))


def test_no_wait_per_chunk_that_is_found():
    """Half of 256 workgroups there: each of them finds more than ten chunks.  Found one per look, at 2048 polls of 0.3 us
    a look, they take ten such waits (over 6 ms); found one after the other, a single wait and the work (under 1 ms)."""
    p = tf.few_problem(16, 1024, 128, 10, 640, 0, "fp8", seed=1)
    P, W = tf.structs(p)
    ws, out = lib.few_workspace(P), torch.empty_like(p.x)
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    ms = []
    with present(128):
        for _ in range(5):
            a.record()
            lib.moe_layer_forward_few(P, W, p.x, out, None, None, ws)
            b.record()
            torch.cuda.synchronize()
            ms.append(a.elapsed_time(b))
    print("[absent] ms with half of the grid:", " ".join(f"{t:.2f}" for t in ms), flush=True)
    assert min(ms) < 3.0
