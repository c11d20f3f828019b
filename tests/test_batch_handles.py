"""Handles of batched calls on the host (no GPU needed): they let go of their tensors
when they are dropped; the caches of one sequence are such handles, too."""
import gc
import weakref

import pytest
import torch


class OnGpu(torch.Tensor):
    """A tensor of the CPU that says it is on a GPU: enough for handles, which only
    keep addresses."""
    is_cuda = True


def gpu(*shape, dtype=torch.int32):
    return torch.zeros(*shape, dtype=dtype).as_subclass(OnGpu)


@pytest.fixture(scope="module")
def s():
    import substitute_speculative_decoding_gb300 as s
    return s


def handles(s):
    shape = (1, 2, 1, 16, 64)
    yield s.paged_kv(gpu(*shape, dtype=torch.bfloat16), gpu(*shape, dtype=torch.bfloat16), gpu(1, 2))
    yield s.paged_kv8(gpu(*shape, dtype=torch.uint8), gpu(*shape, dtype=torch.uint8),
                      gpu(*shape[:4], dtype=torch.float32), gpu(*shape[:4], dtype=torch.float32),
                      gpu(1, 2))
    yield s.batch(gpu(3), gpu(2), 4)


def test_a_dropped_handle_frees_its_tensors_at_once(s):
    gc.collect()
    gc.disable()
    try:
        for h in handles(s):
            kept = [weakref.ref(t) for t in h.keep]
            assert len(kept) >= 2 and all(r() is not None for r in kept)
            del h
            assert [r() for r in kept] == [None] * len(kept)
    finally:
        gc.enable()


def test_a_cache_of_one_sequence_is_a_cache_for_batches(s):
    kv, (k, _, _) = s.make_kv(1, 2, 64, 40, page_size=16, device="cpu")
    one, two = (s.Batch(4096, 4096, n, 4, 0) for n in (1, 2))
    one.device = two.device = k.device
    assert s._same(kv, one) == k.device
    with pytest.raises(s.SubError):
        s._same(kv, two)
    kv.device = torch.device("cuda", 1)
    with pytest.raises(s.SubError):
        s._same(kv, one)
