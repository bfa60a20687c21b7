"""Long read-backs on the GPU: the stored values of every row, by both forms of the kernel, from ragged ranges."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("D,bits", [(128, "84488884"), (64, "48"), (128, "4"), (64, "8888")])
@pytest.mark.parametrize("paged", [False, True], ids=["contiguous", "pages"])
def test_long_read_backs_give_the_stored_values(D, bits, paged):
    from attention_group_quantized_gb300 import kvq
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    Hkv, hb = len(bits), np.array([int(b) for b in bits], np.int8)
    rng = np.random.default_rng(17)
    lens = np.array([0, 1, 5000, 63, 12001, 64, 9000, 20003, 130])
    new = np.minimum(lens, [0, 1, 4000, 63, 12001, 7, 8999, 20003, 130])
    B, pages = len(lens), -(-int(lens.max()) // 64)
    gen = torch.Generator(device="cuda").manual_seed(18)
    if paged:
        table = torch.from_numpy(rng.permutation(B * pages).reshape(B, pages).astype(np.int32)).cuda()
        cache = kvq.empty_page_pool(hb, B * pages, D)
    else:
        cache = kvq.empty_cache(hb, B, pages * 64, D)
    cache.codes.random_(0, 256, generator=gen)
    scale = torch.rand(cache.sz.shape, generator=gen, device="cuda").half().view(torch.int16).int() & 0xFFFF
    zero = torch.randint(0, 16, cache.sz.shape, generator=gen, device="cuda").half().view(torch.int16).int()
    cache.sz.copy_(scale | zero << 16)
    start = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")
    d_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    rows, T = int(new.sum()), int(new.sum()) + 77
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    # what is stored, in 64 bits: every row's place, then its codes and words
    seq = torch.from_numpy(np.repeat(np.arange(B), new)).cuda()
    pos = torch.from_numpy(np.concatenate([np.arange(L - n, L) for n, L in zip(new, lens)])).cuda()
    at = (table[seq, pos // 64].long(), pos % 64) if paged else (seq, pos)
    want = torch.empty((rows, Hkv, D), dtype=torch.float64, device="cuda")
    for h in range(Hkv):
        off, R = cache.head_offset(h), D * int(hb[h]) // 8
        c = cache.codes[off:off + cache.B * cache.Tcap * R].view(cache.B, cache.Tcap, R)[at].double()
        if hb[h] == 4:
            c = torch.stack([c % 16, (c / 16).floor()], -1).flatten(1)
        w = cache.sz.view(Hkv, cache.B, cache.Tcap, D // 32)[h][at]
        s, z = ((w & 0xFFFF).to(torch.int16).view(torch.float16).double().repeat_interleave(32, 1),
                (w >> 16).to(torch.int16).view(torch.float16).double().repeat_interleave(32, 1))
        want[:, h] = (c - z) * s
    for dt, kind in ((torch.float32, kvq.OUT_F32), (torch.bfloat16, kvq.OUT_BF16)):
        out = torch.full((T, Hkv, D), 5.0, dtype=dt, device="cuda")
        tab = (table,) if paged else ()
        (kvq.dequantize_paged if paged else kvq.dequantize)(cache, *tab, start, d_lens, T, out=out, out_dtype=kind,
                                                            status=status)
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        assert torch.equal(out[:rows], want.float().to(dt))      # exact in fp32 (9 + 11 bits), then one rounding
        assert (out[rows:] == 5.0).all()
