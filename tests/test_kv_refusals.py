"""What the key-value cache entry points refuse, through the C ABI and
without a GPU: every refusal comes back before anything is enqueued."""

import ctypes
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "post_weight_quantization_17_amd", "libgptq_mi355x.so")
OK, BAD, WORKSPACE = 0, 1, 3
P = 0x10000  # a pointer that is never followed

i64, vp, ci = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int


class Cache(ctypes.Structure):
    _fields_ = [(n, vp) for n in ("k_codes", "v_codes", "k_grid", "v_grid")] + [
        (n, i64) for n in ("n_pages", "page_size", "kv_heads", "head_dim")] + [("bits", ci)]


class Batch(ctypes.Structure):
    _fields_ = [("table", vp), ("ld_table", i64), ("max_pages", i64), ("lens", vp), ("starts", vp), ("batch", i64),
                ("n_tokens", i64)]


CACHE = dict(k_codes=P, v_codes=P, k_grid=P, v_grid=P, n_pages=10, page_size=64, kv_heads=2, head_dim=128, bits=4)
BATCH = dict(table=P, ld_table=4, max_pages=4, lens=P, starts=None, batch=3, n_tokens=3)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(LIB):
        pytest.fail("libgptq_mi355x.so is not built (run __graft_entry__.build())")
    L = ctypes.CDLL(LIB)
    L.gptq_kv_attention_workspace_size.restype = ctypes.c_size_t
    L.gptq_kv_attention.argtypes = [vp, vp, vp, ci, i64, i64, ctypes.c_double, vp, vp, ci, i64, vp, ctypes.c_size_t, vp, vp]
    for f in (L.gptq_kv_cache_write, L.gptq_kv_cache_read):
        f.argtypes = [vp, vp, vp, vp, ci, i64, i64, vp, vp]
    L.gptq_kv_attention_workspace_size.argtypes = [vp, vp, i64]
    return L


def structs(cache, batch):
    c = None if cache is None else ctypes.byref(Cache(**{**CACHE, **cache}))
    b = None if batch is None else ctypes.byref(Batch(**{**BATCH, **batch}))
    return c, b


def dense(lib, cache=(), batch=(), k=P, v=P, dtype=0, ld=256, ldv=None):
    c, b = structs(cache if cache is None else dict(cache), batch if batch is None else dict(batch))
    ldv = ld if ldv is None else ldv
    st = {f(c, b, k, v, dtype, ld, ldv, None, None) for f in (lib.gptq_kv_cache_write, lib.gptq_kv_cache_read)}
    assert len(st) == 1
    return st.pop()


def attend(lib, cache=(), batch=(), q=P, q_dtype=0, heads=4, ldq=512, scale=0.1, slopes=None, out=P, out_dtype=0, ldo=512,
           ws=P, ws_bytes=1 << 40):
    c, b = structs(cache if cache is None else dict(cache), batch if batch is None else dict(batch))
    return lib.gptq_kv_attention(c, b, q, q_dtype, heads, ldq, scale, slopes, out, out_dtype, ldo, ws, ws_bytes, None, None)


SHARED = [
    (None, {}), ({}, None),
    *[({n: None}, {}) for n in ("k_codes", "v_codes", "k_grid", "v_grid")],
    *[({n: P + 4}, {}) for n in ("k_codes", "v_codes", "k_grid", "v_grid")],
    *[({"bits": b}, {}) for b in (0, 2, 3, 5, 16, -4)],
    *[({"head_dim": d}, {}) for d in (0, 8, 24, 100, 272, -128)],
    *[({"page_size": s}, {}) for s in (0, 8, 15, 48, 2048, -64)],
    *[({"n_pages": n}, {}) for n in (0, -1, 2**31)],
    *[({"kv_heads": n}, {}) for n in (0, -2, 65536)],
    *[({}, {"batch": n, "n_tokens": n}) for n in (-1, 2**25 + 1)],
    *[({}, {"max_pages": n, "ld_table": n}) for n in (0, -1, 2**31)],
    ({}, {"ld_table": 3}), ({}, {"table": None}), ({}, {"lens": None}), ({}, {"n_tokens": 4}), ({}, {"n_tokens": 2}),
    ({}, {"starts": P, "n_tokens": -1}),
]


@pytest.mark.parametrize("case", range(len(SHARED)))
def test_shared_refusals(lib, case):
    cache, batch = SHARED[case]
    assert dense(lib, cache, batch) == BAD
    assert attend(lib, cache, batch) == BAD
    c, b = structs(cache, batch)
    assert lib.gptq_kv_attention_workspace_size(c, b, 4) == 0


def test_dense_refusals(lib):
    for kw in (dict(k=None), dict(v=None), dict(k=P + 1), dict(v=P + 1), dict(dtype=3), dict(dtype=-1), dict(ld=255),
               dict(ldv=255), dict(ld=2**41), dict(dtype=1, k=P + 2)):
        assert dense(lib, **kw) == BAD, kw


def test_attention_refusals(lib):
    inf, nan = float("inf"), float("nan")
    for kw in (dict(q=None), dict(out=None), dict(q=P + 1), dict(out=P + 1), dict(q_dtype=3), dict(out_dtype=-1),
               dict(heads=0), dict(heads=3), dict(heads=-2), dict(heads=65536), dict(ldq=511), dict(ldo=511),
               dict(ldq=2**41), dict(slopes=P + 2), dict(scale=inf), dict(scale=nan), dict(scale=1e39),
               dict(q_dtype=1, q=P + 2)):
        assert attend(lib, **kw) == BAD, kw
    # more workgroups than a launch holds
    assert attend(lib, cache={"kv_heads": 1, "head_dim": 16}, batch={"batch": 2**25, "n_tokens": 2**25}, heads=1, ldq=16,
                  ldo=16) == BAD
    # the same for prompts, whose workgroups are twice as large: 2^23 blocks of 128 rows
    assert attend(lib, cache={"kv_heads": 1, "head_dim": 16}, batch={"starts": P, "batch": 1, "n_tokens": 2**24}, heads=64,
                  ldq=1024, ldo=1024) == BAD


def test_workspace_refusals(lib):
    # one sequence whose table reaches 1024 keys: the keys may be split
    big = {"ld_table": 16, "max_pages": 16}
    c, b = structs({}, big)
    need = lib.gptq_kv_attention_workspace_size(c, b, 4)
    assert need > 0
    assert attend(lib, batch=big, ws_bytes=need - 1) == WORKSPACE
    assert attend(lib, batch=big, ws=None, ws_bytes=need) == BAD
    assert attend(lib, batch=big, ws=P + 8, ws_bytes=need) == BAD
    # 256 keys at most: one unit a row block, no workspace
    c, b = structs({}, {})
    assert lib.gptq_kv_attention_workspace_size(c, b, 4) == 0
    # the size depends on the shapes only
    c, b = structs({}, dict(big, lens=2 * P, table=3 * P))
    assert lib.gptq_kv_attention_workspace_size(c, b, 4) == need


def test_workspace_size_of_refused_head_counts(lib):
    c, b = structs({}, {"ld_table": 2**20, "max_pages": 2**20})
    assert lib.gptq_kv_attention_workspace_size(c, b, 65534) > 0
    for heads in (0, -2, 3, 65536, 2**33):
        assert lib.gptq_kv_attention_workspace_size(c, b, heads) == 0, heads


def test_empty_calls_do_nothing(lib):
    none = {"batch": 0, "n_tokens": 0, "table": None, "lens": None}
    assert dense(lib, batch=none, k=None, v=None) == OK
    assert attend(lib, batch=none, q=None, out=None) == OK
    assert attend(lib, batch={"starts": P, "n_tokens": 0}, q=None, out=None) == OK
    assert dense(lib, batch={"starts": P, "n_tokens": 5, "batch": 0}) == OK
