"""gdn_paged_append and gdn_paged_attn on every route of a call: both attention
kernels, a table that fits its sequences and one with room for many more keys
(the few-row kernel then cuts the list of all keys and joins the pieces through
a workspace). Bounds as derived in test_gpu_paged.py.
"""
import numpy as np
import pytest
import torch

from oracle import paged
from test_gpu_paged import (attend, close, gpu, hidden_values, make, paths,
                            table_of, widen)

pytestmark = pytest.mark.gpu


def tables(s):
    return [s, dict(s, page_table=widen(s["page_table"]))]


# ---- offsets of packed batches -----------------------------------------------
def late(s, before, after):
    """The packed batch with tokens that belong to no sequence around it."""
    q = torch.full((1, before + s["q"].shape[1] + after) + s["q"].shape[2:], 3.0,
                   dtype=s["q"].dtype)
    q[:, before:before + s["q"].shape[1]] = s["q"]
    return dict(s, q=q, cu_seqlens=s["cu_seqlens"] + before)


@pytest.mark.parametrize("hq,hkv,new,keys", [
    (8, 1, (100, 30), (140, 200)), (4, 2, (300, 0, 1), (700, 5, 90)),
    (2, 1, (1, 2, 1), (40, 300, 17)), (3, 3, (0, 0, 70, 5), (9, 0, 70, 5))])
def test_offsets_that_start_late(lib, cuda_device, hq, hkv, new, keys):
    """Tokens before the first sequence and past the last are left alone, and
    those between come out as without them, to the bit where the kernel's cut of
    the keys does not go by the number of tokens."""
    s = make(41, hq=hq, hkv=hkv, new=new, keys=keys, packed=True)
    T = sum(new)
    for wide, t in enumerate(tables(s)):
        x = late(t, 1000, 77)
        for path in paths(lib):
            o, lse = attend(lib, cuda_device, x, path=path)
            ref = attend(lib, cuda_device, t, path=path)
            close(t, ref)
            assert torch.isnan(o[:, :1000]).all() and torch.isnan(o[:, 1000 + T:]).all()
            if path == lib.GDN_PAGED_TILES or (path == lib.GDN_PAGED_ROWS and wide):
                assert torch.equal(o[:, 1000:1000 + T], ref[0])
                assert torch.equal(lse[:, 1000:1000 + T], ref[1])
            close(t, (o[:, 1000:1000 + T], lse[:, 1000:1000 + T]))


@pytest.mark.parametrize("cu", [[0, 60, 0, 30], [0, 10, 5, 60], [0, 20, 40, 61],
                                [-1, 20, 40, 60], [0, 20, 1 << 30, 60],
                                [0, -(1 << 31), 40, 60], [60, 40, 20, 0]])
def test_offsets_out_of_order(lib, cuda_device, cu):
    """Offsets that decrease or leave the batch: recorded, no row written."""
    dev = cuda_device
    s = make(42, hq=8, hkv=2, new=(20, 20, 20), keys=(90, 20, 300), packed=True)
    bad = torch.tensor(cu, dtype=torch.int32, device=dev)
    for t in tables(s):
        args = [gpu(t[n], dev) for n in ("q", "k_cache", "v_cache", "page_table",
                                         "kv_lens")]
        for path in paths(lib):
            out = torch.full(t["q"].shape, 7.0, dtype=t["q"].dtype, device=dev)
            lib.gdn_paged_attn(*args, bad, out=out, path=path)
            assert lib.gdn_device_status() == -1
            assert (out == 7.0).all()
        k, v = (t["normal"]((1, 60, 2, 128)).to(dev) for _ in range(2))
        lib.gdn_paged_append(args[0], k, v, *args[1:], bad)
        assert lib.gdn_device_status() == -1
        assert lib.gdn_device_status() == 0


def test_many_offsets_out_of_order(lib, cuda_device):
    """More sequences than the tile kernel stages, the last pair wrong."""
    dev, N = cuda_device, 9000
    s = make(43, hq=2, hkv=1, d=64, new=(1,) * N, keys=(1,) * N, packed=True,
             poison=False)
    args = [gpu(s[n], dev) for n in ("q", "k_cache", "v_cache", "page_table",
                                     "kv_lens", "cu_seqlens")]
    for path in (lib.GDN_PAGED_ROWS, lib.GDN_PAGED_TILES):
        o = lib.gdn_paged_attn(*args, path=path)
        v = args[2][args[3][:, 0].long(), :, 0].expand(-1, 2, -1)
        assert torch.equal(o[0], v)  # (one key each: its value)
        assert lib.gdn_device_status() == 0
    args[5][N] = N - 3
    for path in (lib.GDN_PAGED_ROWS, lib.GDN_PAGED_TILES):
        out = torch.full_like(args[0], 7.0)
        lib.gdn_paged_attn(*args, path=path, out=out)
        assert lib.gdn_device_status() == -1 and (out == 7.0).all()


def test_append_offsets_that_start_late(lib, cuda_device):
    dev = cuda_device
    s = make(44, hq=4, hkv=2, new=(3, 0, 6), keys=(40, 5, 6), packed=True,
             poison=False)
    rope = table_of(64, 64)
    k, v = (s["normal"]((1, 9, 2, 128)) for _ in range(2))
    ref = paged.append(s["q"], k, v, s["k_cache"], s["v_cache"], s["page_table"],
                       s["kv_lens"], s["cu_seqlens"], rope=rope)

    def pad(t):
        x = torch.full((1, 20) + t.shape[2:], 5.0, dtype=t.dtype, device=dev)
        x[:, 4:13] = t.to(dev)
        return x

    kc, vc = s["k_cache"].to(dev), s["v_cache"].to(dev)
    q = pad(s["q"])
    out = torch.full_like(q, 7.0)
    lib.gdn_paged_append(q, pad(k), pad(v), kc, vc, s["page_table"].to(dev),
                         s["kv_lens"].to(dev), s["cu_seqlens"].to(dev) + 4,
                         rope=rope.to(dev), q_out=out)
    assert lib.gdn_device_status() == 0
    assert (out[:, :4] == 7.0).all() and (out[:, 13:] == 7.0).all()
    for x, r in ((out[:, 4:13], ref[0]), (kc, ref[1]), (vc, ref[2])):
        err = np.abs(x.cpu().double().numpy() - r)
        assert (err <= 2.0 ** -8 * np.abs(r) + 2.0 ** -19).all()


# ---- hidden values ------------------------------------------------------------
@pytest.mark.parametrize("bad", [float("nan"), -float("inf")])
@pytest.mark.parametrize("d,dtype", [(64, "bf16"), (64, "f16"), (128, "f16")])
@pytest.mark.parametrize("new,keys,window", [((3,), (200,), 0), ((3,), (200,), 40),
                                             ((150,), (150,), 0),
                                             ((150,), (400,), 60)])
def test_hidden_values_of_both_types(lib, cuda_device, d, dtype, bad, new, keys,
                                     window):
    s = make(45, hq=6, hkv=2, d=d, dtype=dtype, new=new, keys=keys, poison=False)
    for t in tables(s):
        hidden_values(lib, cuda_device, t, bad, new, keys, window)


@pytest.mark.parametrize("d,dtype", [(128, "bf16"), (64, "f16")])
@pytest.mark.parametrize("new,window", [(40, 0), (40, 30000), (3, 0), (3, 30000)])
def test_hidden_values_in_long_caches(lib, cuda_device, new, window, d, dtype):
    """What a hidden value costs does not grow with the cache: 320 sequences on
    the same 70000 keys, so that a block has whole items. (Key by key over the
    whole cache, a thread's dependent loads of 0.3 us alone would take 20 ms an
    item and group of 32 columns; the calls take some 3 ms.)"""
    dev, N, L = cuda_device, 320, 70000
    s = make(46, hq=4, hkv=1, d=d, dtype=dtype, page=256, new=(new,), keys=(L,),
             poison=False)
    x0, page = L - new, 256

    def put(key, col, value):
        at = int(s["page_table"][0, key // page]), 0, key % page
        s["v_cache"][at + (col,)] = value

    t = np.arange(new)
    inf_at, nan_at = x0 + new // 4, x0 + new // 2
    edge = x0 - window + 1 + new // 3  # seen by the tokens up to new // 3
    clean = dict(s, v_cache=s["v_cache"].clone())
    put(inf_at, 7, float("inf"))
    put(nan_at, slice(None), float("nan"))
    sees_inf, sees_nan = x0 + t >= inf_at, x0 + t >= nan_at
    if window:
        put(edge, slice(None), float("nan"))
        sees_nan |= t <= new // 3
    put7 = int(s["page_table"][0, inf_at // page]), 0, inf_at % page, 7
    clean["v_cache"][put7] = 0.0
    ref, rl, mag = (x[0] for x in paged.attend(
        clean["q"], clean["k_cache"], clean["v_cache"], s["page_table"],
        s["kv_lens"], window=window))
    u = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -11
    bound = u * (np.abs(ref) + 1.02 * mag) + 4e-4 * mag
    if dtype == "f16":
        bound = bound + L * 2.0 ** -25 * float(clean["v_cache"].abs().max())
    args = [s["q"].to(dev).expand(N, -1, -1, -1).contiguous(),
            s["k_cache"].to(dev), s["v_cache"].to(dev),
            s["page_table"].to(dev).expand(N, -1).contiguous(),
            s["kv_lens"].to(dev).expand(N).contiguous()]
    for path in ([lib.GDN_PAGED_ROWS, lib.GDN_PAGED_TILES] if new < 10
                 else [lib.GDN_PAGED_TILES]):
        at = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
        for _ in range(2):
            at[0].record()
            o, lse = lib.gdn_paged_attn(*args, window=window, path=path,
                                        return_lse=True)
            at[1].record()
        torch.cuda.synchronize()
        assert lib.gdn_device_status() == 0
        assert at[0].elapsed_time(at[1]) < 30.0
        o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
        assert (np.abs(lse - rl) <= 2e-4 + 1e-6 * np.abs(rl)).all()
        assert np.isnan(o[:, sees_nan]).all()
        some = ~sees_nan & sees_inf
        assert np.isposinf(o[:, some, :, 7]).all()
        o[..., 7][:, some] = ref[some, :, 7]
        rest = ~sees_nan
        assert (np.abs(o - ref)[:, rest] <= bound[rest]).all()


# ---- fp16 weights ---------------------------------------------------------------
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("below", [17.0, 18.0])
def test_small_f16_weights_behind_a_dominant_key(lib, cuda_device, d, below):
    """One key whose score stands far above the others': their many small
    weights count. 304 sequences on the same keys, so that a block has whole
    items and every weight one reference.

    Bound: weights are rounded relative to 2^7 for the largest score, so each is
    off by at most 2^-25 2^-7 of it (or 2^-11 of itself): keys 2^-32 and 2^-11
    of out in all; one rounding of the output (2^-11); scores here are exact to
    2^-20 (a product of two numbers, all others 0)."""
    dev, N, L = cuda_device, 304, 100000
    s = make(47, hq=1, hkv=1, d=d, dtype="f16", page=256, new=(20,), keys=(L,),
             poison=False)
    k = torch.zeros_like(s["k_cache"])
    v = torch.ones_like(s["v_cache"])
    first = int(s["page_table"][0, 0])
    k[first, 0, 3, 0] = below
    v[first, 0, 3] = 0.0
    q = torch.zeros_like(s["q"])
    q[..., 0] = 1.0
    args = [q.to(dev).expand(N, -1, -1, -1).contiguous(), k.to(dev), v.to(dev),
            s["page_table"].to(dev).expand(N, -1).contiguous(),
            s["kv_lens"].to(dev).expand(N).contiguous()]
    for causal in (True, False):
        seen = (np.arange(L - 20, L) + 1 if causal else np.full(20, L)) - 1.0
        small = seen * np.exp(-below)
        ref = (small / (1.0 + small))[None, :, None, None]
        bound = L * 2.0 ** -32 + ref * (2 * 2.0 ** -11 + 2.0 ** -19)
        for path in (lib.GDN_PAGED_ROWS, lib.GDN_PAGED_TILES):
            o = lib.gdn_paged_attn(*args, scale=1.0, causal=causal, path=path)
            assert lib.gdn_device_status() == 0
            err = np.abs(o.double().cpu().numpy() - ref)
            assert (err <= bound).all(), float((err / ref).max())


# ---- huge scores ------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("new,window", [((40,), 0), ((3,), 0), ((40,), 100)])
def test_huge_scores(lib, cuda_device, dtype, new, window):
    """Scores of some 10^11, whose rounding passes the exponentials' range: every
    token takes its best key's value, and its score for the logarithm of the sum.

    Bounds: fp32 scores are off by at most 128 2^-24 sum |q k| scale (the
    tokens' two best scores are further apart, as is checked), so out is the
    best key's value, to the bit, and lse is within that of the score."""
    s = make(48, dtype=dtype, new=new, keys=(700,), poison=False, std=8000.0)
    s["k_cache"] *= 8000.0
    assert torch.isfinite(s["q"]).all() and torch.isfinite(s["k_cache"]).all()
    place = torch.arange(700)
    ids, rows = s["page_table"][0, place // 16].long(), place % 16
    k, v = (s[n][ids, :, rows].double().repeat_interleave(2, 1)
            for n in ("k_cache", "v_cache"))
    q = s["q"][0].double()
    score = torch.einsum("thd,khd->thk", q, k) * 64.0
    off = torch.einsum("thd,khd->thk", q.abs(), k.abs()) * 64.0 * 128 * 2.0 ** -24
    x = torch.arange(700 - new[0], 700)[:, None]
    sees = (place <= x) & ((place > x - window) if window else (place >= 0))
    score.masked_fill_(~sees[:, None], float("-inf"))
    best = score.topk(2, -1)
    assert (best.values[..., 0] - best.values[..., 1] > 4 * off.amax(-1)).all()
    ref = torch.gather(v.transpose(0, 1), 1, best.indices[..., :1].transpose(0, 1)
                       .expand(-1, -1, 128)).transpose(0, 1)
    for t in tables(s):
        for path in paths(lib):
            o, lse = attend(lib, cuda_device, t, scale=64.0, window=window, path=path)
            assert torch.equal(o[0].cpu().double(), ref)
            err = (lse[0].cpu().double() - best.values[..., 0]).abs()
            assert (err <= off.amax(-1) + 1e-6 * best.values[..., 0].abs()).all()


def test_empty_batch(lib, cuda_device):
    dev = cuda_device
    s = make(49, new=(1,), keys=(20,))
    kc, vc = s["k_cache"].to(dev), s["v_cache"].to(dev)
    table = torch.empty((0, 4), dtype=torch.int32, device=dev)
    lens = torch.empty((0,), dtype=torch.int32, device=dev)
    q = torch.empty((0, 2, 4, 128), dtype=torch.bfloat16, device=dev)
    for path in paths(lib):
        o, lse = lib.gdn_paged_attn(q, kc, vc, table, lens, path=path,
                                    return_lse=True)
        assert o.shape == q.shape and lse.shape == q.shape[:3]
    assert lib.gdn_paged_append(q, q[:, :, :2], q[:, :, :2], kc, vc, table,
                                lens).shape == q.shape
    assert lib.gdn_device_status() == 0


# ---- the cut list of the few-row kernel, and whatever else wide tables reach -----
def check_wide(lib, dev, s, **kw):
    t = tables(s)[1]
    for path in paths(lib):
        close(t, attend(lib, dev, t, path=path, **kw), **kw)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("keys", [1, 16, 63, 65, 129, 700, 3000])
def test_wide_decode_lengths(lib, cuda_device, d, dtype, keys):
    check_wide(lib, cuda_device, make(50, d=d, dtype=dtype, new=(1,), keys=(keys,)))


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("layout", ["hnd", "nhd", "joint"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_wide_pages_and_strides(lib, cuda_device, page, layout, dtype):
    s = make(51, page=page, layout=layout, dtype=dtype, new=(3, 3), keys=(900, 131))
    check_wide(lib, cuda_device, s)


@pytest.mark.parametrize("window", [0, 1, 40, 1000])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("new,keys", [((2, 2), (700, 90)), ((5, 5), (3, 0)),
                                      ((70, 70), (200, 90))])
def test_wide_masks(lib, cuda_device, window, causal, new, keys):
    check_wide(lib, cuda_device, make(52, hq=6, hkv=2, new=new, keys=keys),
               causal=causal, window=window)


def test_wide_mix_of_few_and_many_rows(lib, cuda_device):
    """Few rows on the average, some sequences with many, idle ones between: in
    an automatic packed call each kernel takes its own."""
    s = make(53, hq=2, hkv=1, new=(1, 2, 0, 70, 1, 1) + (1,) * 30,
             keys=(50, 17, 9, 400, 1, 160) + tuple(range(3, 33)))
    check_wide(lib, cuda_device, s)
    s = make(53, hq=6, hkv=2, dtype="f16", new=(0, 1, 130, 0, 7, 33, 0),
             keys=(50, 17, 400, 0, 7, 160, 3))
    check_wide(lib, cuda_device, s)


def test_wide_strided_queries(lib, cuda_device):
    s = make(54, new=(3, 3), keys=(900, 60))
    fused = torch.zeros(2, 3, 8, 128, dtype=torch.bfloat16)
    fused[:, :, :4] = s["q"]
    x = fused.to(cuda_device)
    for t in tables(s):
        args = [gpu(t[n], cuda_device) for n in ("k_cache", "v_cache", "page_table",
                                                 "kv_lens")]
        for path in paths(lib):
            close(t, lib.gdn_paged_attn(x[:, :, :4], *args, path=path,
                                        return_lse=True))


@pytest.mark.parametrize("new,keys", [((1,) * 9, (900, 33, 512, 7, 64, 3000, 5, 300, 77)),
                                      ((90,) * 3, (3000, 90, 500))])
def test_same_bits_on_every_route(lib, cuda_device, new, keys):
    """Twice, and on another stream, where pieces are joined through a workspace
    and where they are not."""
    s = make(55, new=new, keys=keys)
    side = torch.cuda.Stream(cuda_device)
    for t in tables(s):
        for path in paths(lib):
            a = attend(lib, cuda_device, t, path=path)
            b = attend(lib, cuda_device, t, path=path)
            side.wait_stream(torch.cuda.current_stream(cuda_device))
            c = attend(lib, cuda_device, t, path=path, stream=side)
            for x in (b, c):
                assert torch.equal(a[0], x[0]) and torch.equal(a[1], x[1])


def test_bad_lengths_and_pages_on_every_route(lib, cuda_device):
    """A sequence whose keys do not fit its table is skipped, a page outside the
    pool reads as zeros; the others are right."""
    dev = cuda_device
    for new in ((1, 1), (40, 40)):
        s = make(56, new=new, keys=(140, 160))
        ref, _, mag = paged.attend(s["q"], s["k_cache"], s["v_cache"],
                                   s["page_table"], s["kv_lens"])
        for t in tables(s):
            width = t["page_table"].shape[1]
            for path in paths(lib):
                def run(table, lens):
                    out = torch.full(t["q"].shape, 7.0, dtype=torch.bfloat16,
                                     device=dev)
                    lib.gdn_paged_attn(t["q"].to(dev), t["k_cache"].to(dev),
                                       t["v_cache"].to(dev), table.to(dev),
                                       lens.to(dev), out=out, path=path)
                    assert lib.gdn_device_status() == -1
                    return out.float().cpu().numpy()

                for bad in (-1, 16 * width + 1):
                    lens = t["kv_lens"].clone()
                    lens[0] = bad
                    o = run(t["page_table"], lens)
                    assert (o[0] == 7.0).all()
                    assert (np.abs(o[1] - ref[1]) <= 2 ** -6 * mag[1] + 1e-30).all()
                for bad in (-1, t["k_cache"].shape[0]):
                    table = t["page_table"].clone()
                    table[0, 1] = bad
                    o = run(table, t["kv_lens"])
                    assert np.isfinite(o[0]).all()
                    assert (np.abs(o[1] - ref[1]) <= 2 ** -6 * mag[1] + 1e-30).all()


# ---- graphs -------------------------------------------------------------------------
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("new", [1, 2, 40])
def test_every_route_in_a_graph(lib, cuda_device, wide, new):
    """Append and attention captured once and replayed as the sequences grow, on
    each kernel: workspace, cut list, joined pieces and all."""
    dev = cuda_device
    s = make(57, page=64, new=(new,) * 3, keys=(new + 14, new + 31, new + 800),
             poison=False)
    # a page more for each to grow into (of a pool of its own)
    pages = [-(-int(k) // 64) + 1 for k in s["kv_lens"]]
    table = torch.full((3, 200 if wide else max(pages)), -7, dtype=torch.int32)
    order = torch.randperm(sum(pages), generator=torch.Generator().manual_seed(1))
    for i, n in enumerate(pages):
        table[i, :n] = order[sum(pages[:i]):sum(pages[:i]) + n].to(torch.int32)
    shape = (sum(pages),) + s["k_cache"].shape[1:]
    kc, vc = s["normal"](shape).to(dev), s["normal"](shape).to(dev)
    rope = table_of(1100, 128).to(dev)
    table, lens = table.to(dev), s["kv_lens"].to(dev)
    x = s["normal"]((3, new, 8, 128)).to(dev)
    for path in paths(lib):
        def step():
            q = lib.gdn_paged_append(x[:, :, :4], x[:, :, 4:6], x[:, :, 6:], kc,
                                     vc, table, lens, rope=rope)
            return lib.gdn_paged_attn(q, kc, vc, table, lens, return_lse=True,
                                      path=path)

        lens.copy_(s["kv_lens"])
        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
        for _ in range(3):
            lens += 1 if new == 1 else 7
            x.copy_(s["normal"]((3, new, 8, 128)))
            graph.replay()
            torch.cuda.synchronize()
            got = [t.clone() for t in out]
            want = step()
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
            ref, rl, mag = paged.attend(
                lib.gdn_paged_append(x[:, :, :4], x[:, :, 4:6], x[:, :, 6:], kc, vc,
                                     table, lens, rope=rope), kc, vc, table, lens)
            err = np.abs(got[0].double().cpu().numpy() - ref)
            assert (err <= 2.0 ** -8 * (np.abs(ref) + 1.02 * mag) + 4e-4 * mag).all()
    assert lib.gdn_device_status() == 0


# ---- the few-row kernel's choice ------------------------------------------------------
@pytest.mark.parametrize("tokens,users,keys,launches", [
    (1, 1, 2560, 1), (1, 1, 2576, 2), (1, 1, 4096, 2),   # CTAs idle: to 320 each
    (1, 4, 4096, 1), (1, 4, 4112, 2),                    # few idle: to 512 each
    (5, 1, 4096, 1), (5, 1, 4112, 2)])                   # or the tiles
def test_which_calls_are_split(lib, cuda_device, tokens, users, keys, launches):
    """Short tables take one launch, longer ones a second that joins pieces: by
    what the table can hold, the CTAs left over and the rows."""
    dev = cuda_device
    if torch.cuda.get_device_properties(dev).multi_processor_count != 152:
        pytest.skip("the limits below are those of 152 SMs")
    s = make(58, hq=32, hkv=8, new=(tokens,) * users, keys=(30,) * users)
    table = torch.full((users, keys // 16), -7, dtype=torch.int32)
    table[:, :2] = s["page_table"][:, :2]
    t = dict(s, page_table=table)
    before = lib.kernel_counters()
    got = attend(lib, dev, t)
    assert lib.kernel_counters() - before == launches
    close(t, got)
