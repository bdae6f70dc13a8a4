"""Host-only checks of the paged cache's further calls: what the C entry
points refuse (no call here gets as far as a launch), and the index arithmetic
of windows and pages compiled for the host."""
import ctypes
import math

import pytest
import torch

import mhc_hyper_connection_pre_gb300 as mhc
from mhc_hyper_connection_pre_gb300 import build as mbuild
from mhc_hyper_connection_pre_gb300 import kv as kvmod

OK, INVALID, UNSUPPORTED, CUDA_ERR = 0, 1, 2, 3
FAKE = 0x10000000000     # never dereferenced
ROW = (40 + 16) * 128
QKV = FAKE + (4 << 32)
NO_DEVICE = pytest.mark.skipif(torch.cuda.is_available(), reason="a well-formed call would be launched")


@pytest.fixture(scope="module")
def lib():
    mbuild.build()
    return mhc.load_library()


def _cache(**kw):
    a = dict(k=FAKE, v=FAKE + (1 << 32), k_scale=FAKE + (2 << 32), v_scale=FAKE + (3 << 32), num_pages=100, heads=8,
             page_tokens=64, head_dim=128)
    a.update(kw)
    return kvmod._Cache(*a.values())


# -------------------------------------------------------------------- norms ---

def _append_norm(lib, cache=None, **kw):
    a = dict(k=QKV + 40 * 256, k_stride=ROW, v=QKV + 48 * 256, v_stride=ROW, q=QKV, q_stride=ROW, q_heads=40,
             q_out=FAKE + (5 << 32), q_out_stride=40 * 128, q_norm=FAKE + (12 << 32), q_norm_stride=0,
             k_norm=FAKE + (13 << 32), k_norm_stride=128, eps=1e-6, cos=FAKE + (6 << 32), sin=FAKE + (7 << 32),
             rope_rows=1000, rotary_dim=128, interleaved=0, table=FAKE + (8 << 32), width=10, lens=FAKE + (9 << 32),
             cu=None, B=16, T=16, stream=None)
    a.update(kw)
    return lib.mhc_kv_append_norm(cache if cache is not None else _cache(), *a.values())


NORMS = [
    (dict(eps=0.0), INVALID), (dict(eps=-1e-6), INVALID), (dict(eps=1e-21), INVALID), (dict(eps=math.inf), INVALID),
    (dict(eps=math.nan), INVALID), (dict(q_norm=FAKE + (12 << 32) + 8), INVALID),
    (dict(k_norm=FAKE + (13 << 32) + 2), INVALID), (dict(q_norm_stride=120), INVALID),
    (dict(k_norm_stride=132), INVALID), (dict(k_norm_stride=-128), INVALID), (dict(k_norm_stride=1 << 31), INVALID),
    (dict(q=None, q_out=None), INVALID),                           # q_norm without q
    (dict(q_norm=FAKE + (5 << 32)), INVALID),                      # weights that the call writes over
    (dict(k_norm=FAKE + (2 << 32)), INVALID), (dict(k_norm=FAKE + 4096), INVALID),
    (dict(q_norm=FAKE + (5 << 32) - 39 * 256, q_norm_stride=128), INVALID),    # the last head's
    (dict(k=None), INVALID), (dict(T=17), INVALID), (dict(rotary_dim=24), UNSUPPORTED), (dict(T=-1), INVALID),
    (dict(T=0, B=0, k=None, q=None, q_out=None, q_norm=None, cu=FAKE), OK),
]


@pytest.mark.parametrize("case", range(len(NORMS)))
def test_append_norm_refuses(lib, case):
    kw, status = NORMS[case]
    assert _append_norm(lib, **kw) == status


@NO_DEVICE
def test_append_norm_passes_the_checks(lib):
    """With no device in the process well-formed calls end as MHC_ERR_CUDA."""
    assert _append_norm(lib) == CUDA_ERR
    assert _append_norm(lib, q_norm=None) == CUDA_ERR
    assert _append_norm(lib, k_norm=None) == CUDA_ERR
    assert _append_norm(lib, q=None, q_out=None, q_norm=None) == CUDA_ERR
    assert _append_norm(lib, q_norm=None, k_norm=None, eps=0.0) == CUDA_ERR       # no norm: eps is not read
    assert _append_norm(lib, q_norm=FAKE + (5 << 32) - 40 * 256, q_norm_stride=128) == CUDA_ERR      # just before q_out


@pytest.mark.parametrize("call", ["k", "v"])
def test_queries_in_place_are_not_keys_or_values_too(lib, call):
    """q_out may be q, but then no other input may lie there."""
    assert _append_norm(lib, q_out=QKV, q_out_stride=ROW, q_norm=None, k_norm=None, **{call: QKV}) == INVALID
