"""Host-side argument checks, without a GPU, of verification against probability
rows, the 4-bit LM head and the page cache."""
import ctypes
import os

import pytest
import torch

from speculative_decoding_verification_pipeline_amd import sampler as SM
from speculative_decoding_verification_pipeline_amd.cache import PageCache


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(SM.LIB_PATH):
        from speculative_decoding_verification_pipeline_amd import build
        build.build()
    return SM.load_library()


def test_calls_reject_null_handles(lib):
    bad = SM.SS_ERR_INVALID_ARG
    t = SM.CBlockTables()
    assert lib.ss_spec_verify_probs(None, None, 0, 0, None, 0, None, None, None, 1, 1, None, None,
                                    None, None) == bad
    assert lib.ss_lmhead_quant_logits(None, None, None, None, 2, None, 64, 1, None, 0, 0,
                                      None) == bad
    assert lib.ss_cache_reserve(None, ctypes.byref(t), None, None, 1, None, None) == bad
    assert lib.ss_cache_fork(None, ctypes.byref(t), None, None, 1, None, None) == bad
    assert lib.ss_cache_commit(None, ctypes.byref(t), None, None, 0, 0, None, 1, 1, None, None) == bad
    assert lib.ss_cache_truncate(None, ctypes.byref(t), None, None, 1, None) == bad
    assert lib.ss_cache_copy_pages(None, None, None, None, 1, None, None) == bad
    assert lib.ss_cache_workspace_bytes(None) == 0
    lib.ss_cache_destroy(None)


GOOD = dict(num_planes=2, num_pages=8, page_size=4, heads=2, piece_bytes=16, page_stride=128,
            slot_stride=32, head_stride=16, max_batch=3, max_blocks=5, device=0)


@pytest.mark.parametrize("change", [
    {"num_planes": 0}, {"num_planes": 4097}, {"num_pages": 0}, {"num_pages": 4194305},
    {"page_size": 0}, {"page_size": 65537}, {"heads": 0}, {"heads": 65537}, {"piece_bytes": 0},
    {"piece_bytes": 1 << 24}, {"max_batch": 0}, {"max_batch": 65536}, {"max_blocks": 0},
    {"max_blocks": 1 << 29}, {"device": -1}, {"page_stride": 0}, {"slot_stride": -32},
    {"head_stride": 15}, {"slot_stride": 31}, {"page_stride": 127}, {"page_stride": 32},
    {"max_batch": 65535, "max_blocks": 65535}, {"page_size": 4096, "max_blocks": 1 << 20},
    {"page_stride": 1 << 60},
    {"num_planes": 4096, "heads": 1024, "piece_bytes": 1024, "page_size": 1, "num_pages": 1,
     "head_stride": 1024},
])
def test_cache_create_rejects_bad_shapes_before_touching_hip(lib, change):
    cfg = SM.CacheConfig(**{**GOOD, **change})
    planes = (ctypes.c_void_p * 4097)(*range(64, 64 * 4098, 64))
    h = ctypes.c_void_p()
    assert lib.ss_cache_create(ctypes.byref(cfg), planes, ctypes.byref(h)) == SM.SS_ERR_INVALID_ARG
    assert not h.value


def test_cache_create_rejects_null_pointers(lib):
    cfg = SM.CacheConfig(**GOOD)
    planes = (ctypes.c_void_p * 2)(64, None)
    h = ctypes.c_void_p()
    for c, p, o in ((None, planes, ctypes.byref(h)), (ctypes.byref(cfg), None, ctypes.byref(h)),
                    (ctypes.byref(cfg), planes, None), (ctypes.byref(cfg), planes, ctypes.byref(h))):
        assert lib.ss_cache_create(c, p, o) == SM.SS_ERR_INVALID_ARG


def test_cache_create_rejects_a_plane_named_twice(lib):
    cfg = SM.CacheConfig(**{**GOOD, "num_planes": 3})
    h = ctypes.c_void_p()
    for at in ([4096, 8192, 4096], [64, 64, 128]):
        planes = (ctypes.c_void_p * 3)(*at)
        assert lib.ss_cache_create(ctypes.byref(cfg), planes, ctypes.byref(h)) == SM.SS_ERR_INVALID_ARG
        assert not h.value


def test_page_cache_takes_device_planes_only(lib):
    for planes in ([], [torch.zeros(2, 4, 1, 8)], torch.zeros(2, 2, 4, 1, 8)):
        with pytest.raises(ValueError):
            PageCache(planes, 2, 2)


def test_row_stride():
    x = torch.empty(3, 4, 10)
    assert SM._row_stride(x, "x") == 10
    assert SM._row_stride(x[:, :, :7], "x") == 10
    assert SM._row_stride(x[:1, 1:3], "x") == 10
    assert SM._row_stride(torch.empty(5, 0, 10), "x") == 10
    assert SM._row_stride(torch.empty(5, 20)[:, None, :10], "x") == 20
    for bad in (x[:, :3], x.transpose(1, 2), x[:, :, ::2], x[:1, :1].expand(3, 4, 10),
                x.transpose(0, 1)):
        with pytest.raises(ValueError):
            SM._row_stride(bad, "x")


def test_commit_with_verdicts_rejects_a_null_handle(lib):
    t = SM.CBlockTables()
    assert lib.ss_cache_commit_reserved(None, ctypes.byref(t), None, None, 0, 0, None, 1, 1, None, None,
                                        None) == SM.SS_ERR_INVALID_ARG
    assert "ss_cache_commit_reserved" in SM.EXPORTED
