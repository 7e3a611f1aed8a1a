"""The operators of a serving step in a row, as a layer with self and cross
attention runs them: the batch's tables, the normed and turned heads into the
cache, attention to the own cache (a chunk, then single tokens), the queries of
the cross layer, attention to an encoder's states; against 64-bit arithmetic on
the oracle's caches."""
import numpy as np
import pytest
import torch

import oracle
from tests import gpu_helpers as gh
from tests import step_reference as ref

pytestmark = pytest.mark.gpu

pq = pytest.importorskip("paged_quantized_kv_cache_b200")


@pytest.mark.parametrize("kv_dtype,dtype", [(pq.BF16, torch.bfloat16), (pq.FP8_E4M3, torch.bfloat16),
                                            (pq.FP4_E2M1, torch.float16)], ids=["bf16", "fp8", "fp4"])
def test_chunk_then_decode_steps(kv_dtype, dtype):
    Hq, Hkv, D, B, most, nb = 8, 2, 128, 3, 8, 40
    rng = np.random.default_rng(7)
    pool = pq.BlockPool(nb)
    g, o = gh.new_pair(kv_dtype, nb, Hkv, D)
    i32 = lambda x: torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()  # noqa: E731
    tables, host_tables = torch.full((B, most), -1, dtype=torch.int32, device="cuda"), np.full((B, most), -1)
    # the encoder's states: written once, in the same pool
    enc = [70, 33, 0]
    enc_rows = np.full((B, 5), -1)
    for b, L in enumerate(enc):
        if L:
            enc_rows[b, :-(-L // 16)] = pool.alloc(-(-L // 16))
            k, v = (torch.from_numpy(rng.standard_normal((L, Hkv, D))).to(dtype) for _ in range(2))
            p = np.arange(L)
            assert gh.write_both(g, o, k, v, enc_rows[b][p // 16] * 16 + p % 16) == (0, 0)
    angle = np.arange(200)[:, None] * 1000.0 ** (-np.arange(D // 2) / (D // 2))
    table = torch.from_numpy(np.concatenate([np.cos(angle), np.sin(angle)], 1)).float()
    rotary = pq.Rotary(table.cuda())
    wq, wk = (torch.from_numpy(1 + 0.1 * rng.standard_normal(D)).float() for _ in range(2))
    scale, start = 1 / np.sqrt(D), np.zeros(B, np.int64)
    for new in ([40, 17, 9], [1, 1, 1], [1, 1, 1]):
        new, T, cap = np.array(new), sum(new), sum(new) + 3
        fresh = int((-(-(start + new) // 16) - -(-start // 16)).sum())
        ids = pool.alloc(fresh)
        err = gh.err_flag()
        slots, pos, cu, lens = (torch.empty(n, dtype=torch.int32, device="cuda") for n in (cap, cap, B + 1, B))
        pq.build_batch(i32(start), i32(new), i32(ids), tables, nb, slots, pos, cu, lens, err)
        host_tables, hs, hp, hcu, hl, _ = ref.batch(start, new, ids, host_tables, nb, cap)
        # the padded rows hold anything; their slots are -1
        x = torch.from_numpy(rng.standard_normal((cap, (Hq + 2 * Hkv) * D))).to(dtype)
        gx = x.cuda()
        cut = [t.view(cap, -1, D) for t in gx.split((Hq * D, Hkv * D, Hkv * D), 1)]
        q = torch.empty(cap, Hq, D, dtype=dtype, device="cuda")
        pq.qkv_norm_rope_write(*cut, pos, rotary, q, slots, g, err, q_weight=wq.cuda(), k_weight=wk.cuda())
        out = torch.zeros_like(q)
        if new.max() > 1:
            pq.paged_prefill_attention(q, cu, int(new.max()), g, tables, lens, scale, out, err)
        else:
            ws = pq.decode_workspace(B, Hq, Hkv, D, most)
            pq.paged_decode_attention(q[:B], g, tables, lens, scale, out[:B], ws, err)
        cross_q, cross_out = torch.empty_like(q), torch.zeros_like(q)
        pq.qk_norm_rope(out, None, None, None, cross_q, None, err, q_weight=wq.cuda())
        seen = np.stack([np.zeros(cap), np.full(cap, 50)], 1)
        seen[::4, 1] = 0
        pq.paged_cross_attention(cross_q, cu, int(new.max()), g, i32(enc_rows), i32(enc), scale, cross_out, err,
                                 kv_ranges=i32(seen))
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        np.testing.assert_array_equal(tables.cpu().numpy(), host_tables)
        # queries and keys against 64 bits; the cache's bytes from those keys, by the oracle
        hx = [t.view(cap, -1, D) for t in x.split((Hq * D, Hkv * D, Hkv * D), 1)]
        z, size = ref.norm_rope(hx[0], wq, 1e-6, hp, b"", table, False)
        assert (np.abs(q.double().cpu().numpy() - z) <= ref.rope_tolerance(z, size, dtype)).all()
        keys = torch.empty(cap, Hkv, D, dtype=dtype, device="cuda")
        pq.qk_norm_rope(cut[1], None, pos, rotary, keys, None, err, q_weight=wk.cuda())
        z, size = ref.norm_rope(hx[1], wk, 1e-6, hp, b"", table, False)
        assert (np.abs(keys.double().cpu().numpy() - z) <= ref.rope_tolerance(z, size, dtype)).all()
        assert oracle.kv_cache_write(o, keys.cpu(), hx[2].contiguous(), hs) == 0
        gh.assert_cache_equal(g, o)
        # self attention
        want, rerr = oracle.paged_prefill(o, q[:T].cpu(), hcu, host_tables, hl, scale)
        assert rerr == 0
        gh.assert_close(out[:T], want, kv_dtype, tag="self")
        # cross attention
        want, tol = ref.cross(o, cross_q[:T].cpu(), hcu, enc_rows, enc, scale, seen)
        assert (np.abs(cross_out[:T].double().cpu().numpy() - want) <= tol).all()
        assert (cross_out[T:] == 0).all()
        start += new


def test_calls_refuse_tensors_that_they_do_not_take():
    """Types, shapes, strides and devices that the Python calls refuse, with the outputs left alone."""
    i32 = lambda *n: torch.zeros(*n, dtype=torch.int32, device="cuda")  # noqa: E731
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    err, out = i32(1), torch.full_like(x, 7)
    table = pq.Rotary(torch.zeros(8, 64, device="cuda"))
    p = i32(4)
    c = pq.allocate_cache(pq.BF16, 2, 2, 64)
    bad = [
        lambda: pq.build_batch(i32(2), i32(3), i32(1), i32(2, 4), 9, i32(5), i32(5), i32(3), i32(2), err),
        lambda: pq.build_batch(i32(2), i32(2), i32(1), i32(2, 4), 9, i32(5), i32(4), i32(3), i32(2), err),
        lambda: pq.build_batch(i32(2), i32(2), i32(1), i32(8), 9, i32(5), i32(5), i32(3), i32(2), err),
        lambda: pq.build_batch(i32(2), i32(2).long(), i32(1), i32(2, 4), 9, i32(5), i32(5), i32(3), i32(2), err),
        lambda: pq.build_batch(i32(2), i32(2), i32(1), i32(2, 8)[:, ::2], 9, i32(5), i32(5), i32(3), i32(2), err),
        lambda: pq.build_batch(i32(2), i32(2), i32(1).cpu(), i32(2, 4), 9, i32(5), i32(5), i32(3), i32(2), err),
        lambda: pq.build_batch(i32(2), i32(2), i32(1), i32(2, 4), 2 ** 40, i32(5), i32(5), i32(3), i32(2), err),
        lambda: pq.qk_norm_rope(x, x.half(), p, table, out, out, err),
        lambda: pq.qk_norm_rope(x, None, p, table, out, out, err),
        lambda: pq.qk_norm_rope(x, None, p[:3], table, out, None, err),
        lambda: pq.qk_norm_rope(x, None, None, table, out, None, err),
        lambda: pq.qk_norm_rope(x, None, p, pq.Rotary(table.cos_sin, b"\0"), out, None, err),
        lambda: pq.qk_norm_rope(x, None, p, pq.Rotary(table.cos_sin.double()), out, None, err),
        lambda: pq.qk_norm_rope(x.transpose(0, 1), None, p, table, out.transpose(0, 1), None, err),
        lambda: pq.qk_norm_rope(x, None, p, table, out, None, err, q_weight=torch.ones(63, device="cuda")),
        lambda: pq.qk_norm_rope(x, None, p, table, out, None, err, q_weight=torch.ones(64)),
        lambda: pq.qk_norm_rope(x, None, p, table, out.float(), None, err),
        lambda: pq.qkv_norm_rope_write(x, x, x[:, :1], p, table, out, p, c, err),
        lambda: pq.qkv_norm_rope_write(x, x, x, p, table, out, p[:2], c, err),
        lambda: pq.paged_cross_attention(x, i32(3), 1, c, i32(1, 1), i32(1), 1.0, out, err),
        lambda: pq.paged_cross_attention(x, i32(2), 1, c, i32(1, 1), i32(1), 1.0, out, err, kv_ranges=i32(3, 2)),
        lambda: pq.paged_cross_attention(x, i32(2), "1", c, i32(1, 1), i32(1), 1.0, out, err),
        lambda: pq.paged_cross_attention(x, i32(2), 1, c, i32(1, 1), i32(1), 1.0, out, None),
    ]
    for k, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            raise AssertionError("call %d was taken" % k)
    with pytest.raises(pq.PqkvError):
        pq.paged_cross_attention(x, i32(2), 0, c, i32(1, 1), i32(1), 1.0, out, err)
    torch.cuda.synchronize()
    assert (out == 7).all() and int(err.item()) == 0
    for empty in (pq.qk_norm_rope, None):  # no tokens: nothing to do
        if empty:
            pq.qk_norm_rope(x[:0], x[:0], p[:0], table, out[:0], out[:0], err)
        else:
            pq.paged_cross_attention(x[:0], i32(2), 1, c, i32(1, 1), i32(1), 1.0, out[:0], err)
