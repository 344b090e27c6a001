"""gdn_paged_append and gdn_paged_attn on every route of a call: both attention
kernels, a table that fits its sequences and one with room for many more keys
(the few-row kernel then cuts the list of all keys and joins the pieces through
a workspace). Bounds as derived in test_gpu_paged.py.
"""
import numpy as np
import pytest
import torch

from oracle import paged
from test_gpu_paged import attend, close, gpu, make, paths, table_of, widen

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
