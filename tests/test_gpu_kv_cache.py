"""The quantised key-value cache on the GPU against the oracle (needs an
MI355X): stored codes and grids bit for bit, values read back within their
rounding, attention within the bound of tests/kv_cases.py.
"""

import numpy as np
import pytest
import torch

import oracle.kv_oracle as K
from tests import kv_cases as C

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
TORCH = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def up(a):
    a = np.ascontiguousarray(a)
    return torch.from_numpy(a.view(np.int32) if a.dtype == np.uint32 else a).to(DEV)


def dense(values, name):
    """A device tensor of float values (already of the type's precision)."""
    return torch.from_numpy(np.ascontiguousarray(values, dtype=np.float32)).to(DEV).to(TORCH[name])


def upload(g, cache):
    return g.KVCache(k_codes=up(cache["k_codes"]), v_codes=up(cache["v_codes"]), k_grid=up(cache["k_grid"]),
                     v_grid=up(cache["v_grid"]), head_dim=cache["head_dim"], bits=cache["bits"],
                     info=torch.zeros(1, dtype=torch.int32, device=DEV))


def same_cache(dev, ref):
    for n in ("k_grid", "v_grid", "k_codes", "v_codes"):
        assert np.array_equal(getattr(dev, n).cpu().numpy().view(np.uint32), ref[n]), n


def as64(t):
    return t.float().cpu().numpy().astype(np.float64)


def check_attention(got, qf, cache, table, lens, starts, scale, slopes, qdt, odt):
    ref, mag, _, bad = K.attention(qf, cache, table, lens, starts, scale, slopes)
    bound = C.attention_bound(ref, mag, qf, cache, scale, slopes, qdt, odt, int(max(max(lens), 1)))
    err = np.abs(as64(got) - ref)
    assert np.all(err <= bound), float(np.max(err / bound))
    return bad


# (dim, bits, page, heads, lens, news, dtype, pad of the token stride)
STORE = [
    (128, 4, 16, 32, [778], [1], "f32", 0),
    (128, 8, 64, 8, [1 + 61 * i for i in range(40)], [1] * 40, "bf16", 0),
    (80, 4, 32, 5, [700, 0, 65, 333], [211, 0, 65, 7], "bf16", 0),
    (64, 8, 16, 3, [100, 31], [90, 1], "f16", 4),
    (16, 4, 16, 7, [5, 2, 40], [2, 4, 39], "f32", 1),
    (256, 8, 1024, 2, [1030], [1030], "f16", 0),
    (192, 4, 128, 1, [257], [129], "bf16", 0),
    (112, 8, 256, 2, [300], [299], "f32", 0),
    (32, 4, 16, 1, list(range(1, 131)), [1 + i % 3 for i in range(130)], "f16", 0),
]


@pytest.mark.parametrize("case", range(len(STORE)))
def test_store_and_read_back(gpu, case):
    dim, bits, page, heads, lens, news, dtype, pad = STORE[case]
    rng = np.random.default_rng(case)
    table, lens, starts, n_pages = C.batch(rng, lens, news, page)
    cache = C.cache(rng, n_pages, heads, page, dim, bits, garbage=True)
    n = int(sum(news))
    x = rng.standard_normal((2, n, heads, dim)) * np.exp(rng.standard_normal((2, n, 1, 1)))
    x[0, 0, 0] = 0.0
    x[1, 0, 0] = np.abs(x[1, 0, 0])
    x[0, -1, 0] = rng.integers(-30, 31, dim) / 2.0
    x[1, -1, 0] *= {"f16": 8000, "bf16": 3e37, "f32": 3e37}[dtype]
    x[:, n // 2, 0] *= {"f16": 6e-8, "bf16": 1e-38, "f32": 1e-41}[dtype]
    x = np.clip(x, -6e4, 6e4) if dtype == "f16" else x
    buf = torch.zeros((2, n, heads * dim + pad), dtype=TORCH[dtype], device=DEV)
    kf, vf = (C.cast(a, dtype)[0] for a in x)
    k, v = (buf[i, :, : heads * dim].unflatten(1, (heads, dim)) for i in range(2))
    k.copy_(dense(kf, dtype))
    v.copy_(dense(vf, dtype))
    dev = upload(gpu, cache)
    td, ld, sd = up(table), up(lens), None if starts is None else up(starts)
    gpu.gptq_kv_cache_write(dev, k, v, td, ld, starts=sd)
    ref, _ = K.write(cache, kf.astype(np.float64), vf.astype(np.float64), table, lens, starts)
    same_cache(dev, ref)
    want, _, _ = K.read(ref, table, lens, starts, n)
    for odt in ("f16", "bf16", "f32"):
        got = gpu.gptq_kv_cache_read(dev, td, ld, starts=sd, n_tokens=n, dtype=TORCH[odt])
        for a, w in zip(got, want):
            big = np.abs(w) > {"f16": 65519, "bf16": 3.38e38, "f32": 3.4e38}[odt]
            err = np.abs(as64(a) - w)
            tol = np.abs(w) * (C.EPS[odt] + C.EPS["f32"]) * 1.001 + C.TINY[odt]
            nan = np.isnan(w) & np.isnan(as64(a))  # a vector whose range is not finite
            assert np.all(big | nan | (err <= tol)), float(np.nanmax(np.where(big, 0, err - tol)))
    assert int(dev.info.item()) == 0


# (dim, bits, page, kv heads, query heads, lens, news, q dtype, out dtype, slopes, ragged)
ATTEND = [
    (128, 4, 16, 32, 32, [1], [1], "f32", "f16", False, None),
    (128, 4, 16, 32, 32, [130], [1], "f32", "f16", False, None),
    (128, 4, 64, 8, 64, [4099], [1], "bf16", "bf16", False, None),
    (128, 8, 64, 8, 32, [0, 1, 16, 17, 63, 64, 65, 500, 1500, 2047], [1] * 10, "bf16", "bf16", False, None),
    (128, 8, 64, 2, 2, [3000, 70], [1, 1], "f16", "f16", True, None),
    (80, 8, 32, 4, 4, [901, 0, 31], [1] * 3, "f32", "f32", True, None),
    (80, 4, 256, 2, 10, [300], [1], "f16", "f16", False, None),
    (64, 4, 16, 2, 6, [200, 777], [1, 1], "f16", "f16", False, None),
    (64, 8, 1024, 1, 1, [1025], [1], "bf16", "f32", False, None),
    (16, 8, 16, 3, 3, [100], [1], "f16", "f16", False, None),
    (48, 4, 32, 1, 5, [333], [1], "f32", "bf16", True, None),
    (96, 8, 128, 2, 4, [129, 257], [1, 1], "f16", "bf16", False, None),
    (112, 4, 64, 1, 3, [400], [1], "bf16", "bf16", False, None),
    (192, 8, 16, 1, 2, [222], [1], "f16", "f16", True, None),
    (256, 4, 64, 2, 8, [555, 64], [1, 1], "f16", "f16", False, None),
    (256, 8, 64, 1, 1, [129], [1], "f32", "f32", False, None),
    (128, 4, 16, 1, 20, [300, 5], [1, 1], "bf16", "bf16", False, None),
    # prompts and chunks
    (128, 4, 64, 2, 8, [150, 0, 77, 40], [150, 0, 7, 40], "f16", "f16", False, None),
    (64, 8, 16, 1, 3, [90, 4, 33], [33, 9, 1], "bf16", "bf16", True, None),
    (80, 4, 32, 2, 2, [61], [61], "f32", "f32", False, None),
    (256, 8, 32, 1, 2, [70], [17], "f16", "f16", False, None),
    (128, 8, 16, 1, 1, [40 + i for i in range(70)], [1 + i % 2 for i in range(70)], "f16", "f16", False, None),
    # 64 query rows a sequence or more in the mean: the prompts' kernel
    (128, 8, 16, 2, 2, [333], [333], "bf16", "bf16", False, None),
    (64, 4, 64, 1, 4, [500, 0, 20], [133, 0, 20], "f16", "f16", True, None),
    (64, 8, 16, 3, 3, [130], [129], "f32", "f32", False, None),
    (256, 4, 32, 1, 2, [300], [70], "f16", "f16", False, None),
    (256, 8, 16, 1, 1, [150, 40], [100, 40], "f32", "f16", False, None),
    (80, 8, 128, 2, 6, [90, 200], [90, 1], "bf16", "f16", True, None),
    (112, 4, 16, 1, 1, [257], [190], "f32", "f32", True, None),
    (192, 8, 64, 1, 2, [66, 3], [66, 65], "f16", "bf16", False, None),
    (16, 4, 16, 2, 64, [9], [2], "f16", "f32", False, None),
    (48, 8, 64, 1, 5, [1500], [21], "bf16", "bf16", False, None),
    (128, 4, 64, 1, 4, [3000, 100], [40, 5], "f16", "f16", False, None),
]


@pytest.mark.parametrize("case", range(len(ATTEND)))
def test_attention(gpu, case):
    dim, bits, page, heads, hq, lens, news, qdt, odt, use_slopes, ragged = ATTEND[case]
    rng = np.random.default_rng(100 + case)
    table, lens, starts, n_pages = C.batch(rng, lens, news, page, ragged=ragged)
    cache = C.cache(rng, n_pages, heads, page, dim, bits)
    C.poison(cache, table, lens)
    n = int(sum(news))
    qf, _ = C.cast(1.5 * rng.standard_normal((n, hq, dim)), qdt)
    slopes = (2.0 ** -rng.uniform(1, 8, hq)).astype(np.float32) if use_slopes else None
    dev = upload(gpu, cache)
    args = (dense(qf, qdt), dev, up(table), up(lens))
    kw = dict(starts=None if starts is None else up(starts), slopes=None if slopes is None else up(slopes), dtype=TORCH[odt])
    got = gpu.gptq_kv_attention(*args, **kw)
    again = gpu.gptq_kv_attention(*args, **kw)
    torch.cuda.synchronize()
    assert torch.equal(got, again)  # deterministic
    check_attention(got, qf, cache, table, lens, starts, dim**-0.5, slopes, qdt, odt)
    assert int(dev.info.item()) == 0
