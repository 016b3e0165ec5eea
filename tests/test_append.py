"""vattn_append against a 64-bit append, for every element of the caches."""
import pytest
import torch

from tests.serving import amplitude, frequencies, rotate64
from verified_sparse_attention_b200 import _abi
from verified_sparse_attention_b200.decoder import SparseDecoder
from verified_sparse_attention_b200.rotary import Rotary

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
RANK = 32


# ------------------------------------------------------------ refusals of the wrapper (CPU)
def _fake(proxy="exact", dtype=torch.bfloat16):
    """A decoder without a context: its checks run on host tensors."""
    dec = SparseDecoder.__new__(SparseDecoder)
    dec.device, dec._index, dec._cache_index = torch.device("cpu"), -1, -1
    dec.num_q_heads, dec.num_kv_heads, dec.head_dim, dec.page_size = 8, 2, 64, 16
    dec.max_batch, dec.max_ctx, dec.pages_per_seq, dec.proxy, dec.dtype, dec.ctx = 4, 100, 7, proxy, dtype, None
    dec._cache_shape = (2, 16, 64)
    dec._stream = lambda s: 0
    return dec


def _args(**kw):
    bf = torch.bfloat16
    a = dict(k=torch.zeros(3, 2, 64, dtype=bf), v=torch.zeros(3, 2, 64, dtype=bf),
             k_cache=torch.zeros(5, 2, 16, 64, dtype=bf), v_cache=torch.zeros(5, 2, 16, 64, dtype=bf),
             page_table=torch.zeros(3, 7, dtype=torch.int32), seq_lens=torch.ones(3, dtype=torch.int32), num_pages=5)
    a.update(kw)
    return a


@pytest.mark.parametrize("bad", [
    dict(k=torch.zeros(3, 2, 64)), dict(k=torch.zeros(3, 1, 64, dtype=torch.bfloat16)),
    dict(v=torch.zeros(2, 2, 64, dtype=torch.bfloat16)),
    dict(v=torch.zeros(3, 64, 2, dtype=torch.bfloat16).transpose(1, 2)),
    dict(k=torch.zeros(2, 3, 64, dtype=torch.bfloat16).transpose(0, 1)),
    dict(k_cache=torch.zeros(5, 2, 32, 64, dtype=torch.bfloat16)), dict(num_pages=6),
    dict(v_cache=torch.zeros(5, 2, 64, 16, dtype=torch.bfloat16).transpose(2, 3)),
    dict(page_table=torch.zeros(3, 6, dtype=torch.int32)), dict(page_table=torch.zeros(3, 7)),
    dict(seq_lens=torch.ones(3)), dict(seq_lens=torch.ones(2, dtype=torch.int32)),
    dict(seq_lens=torch.ones(5, dtype=torch.int32), page_table=torch.zeros(5, 7, dtype=torch.int32)),
    dict(cu_tokens=torch.zeros(3, dtype=torch.int32)), dict(cu_tokens=torch.zeros(4)),
    dict(q=torch.zeros(3, 8, 32, dtype=torch.bfloat16)),
    dict(q=torch.zeros(3, 8, 64, dtype=torch.bfloat16), q_out=torch.zeros(3, 8, 64)),
    dict(q=torch.zeros(3, 8, 64, dtype=torch.bfloat16), q_out=torch.zeros(3, 9, 64, dtype=torch.bfloat16)[:, :8]),
    dict(rotary=Rotary(head_dim=128))])
def test_append_wrapper_refusals(bad):
    with pytest.raises(ValueError):
        _fake().append(**_args(**bad))


def test_append_wrapper_refuses_missing_proxy_caches():
    with pytest.raises(ValueError):
        _fake("sparq").append(**_args())
    with pytest.raises(ValueError):
        _fake("loki").append(**_args(k_proj_cache=torch.zeros(5, 2, 16, 32, dtype=torch.bfloat16)))


def test_append_needs_a_context():
    with pytest.raises(_abi.VattnError):   # everything in order but the context
        _fake().append(**_args())


def test_append_wrapper_takes_views_of_a_single_token():
    # a row of a wider tensor is contiguous: as q_out, and in place
    wide = torch.zeros(1, 12, 64, dtype=torch.bfloat16)
    one = dict(k=wide[:, 8:10], v=wide[:, 10:], page_table=torch.zeros(1, 7, dtype=torch.int32),
               seq_lens=torch.ones(1, dtype=torch.int32), q=wide[:, :8])
    for out in (None, wide[:, :8], torch.zeros(1, 9, 64, dtype=torch.bfloat16)[:, 1:]):
        with pytest.raises(_abi.VattnError):   # everything in order but the context
            _fake().append(**_args(**one, q_out=out))


# ------------------------------------------------------------ on the GPU
def _case(*, dtype, d, Hq, Hkv, ps, new, before, proxy, seed=0, wide=False, pad=0, spare=1):
    """One call's tensors: sequence b has before[b] positions and gets new[b] (host tensors)."""
    g = torch.Generator().manual_seed(seed)
    dt, B, T = DT[dtype], len(new), sum(new)
    lens = [a + n if n else a for a, n in zip(before, new)]
    pps = -(-max(max(lens), 1) // ps)
    table = torch.full((B, pps), -1, dtype=torch.int64)
    pages = 0
    for b in range(B):
        n = -(-lens[b] // ps)
        table[b, :n] = torch.arange(pages, pages + n)
        pages += n
    pages += spare
    perm = torch.randperm(pages, generator=g)
    table = torch.where(table >= 0, perm[table.clamp_min(0)], table)

    def randn(*s):
        return torch.randn(*s, generator=g).to(dt)

    rows = T + pad
    if wide:
        x = randn(rows, Hq + 2 * Hkv + 1, d)
        q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:Hq + 2 * Hkv]
    else:
        q, k, v = randn(rows, Hq, d), randn(rows, Hkv, d), randn(rows, Hkv, d)
    c = dict(q=q, k=k, v=v, page_table=table.int(), seq_lens=torch.tensor(lens, dtype=torch.int32),
             cu_tokens=torch.tensor([0] + new).cumsum(0).int(), num_pages=pages,
             k_cache=randn(pages, Hkv, ps, d), v_cache=randn(pages, Hkv, ps, d),
             k_t_cache=randn(pages, Hkv, d, ps) if proxy == "sparq" else None,
             k_proj_cache=randn(pages, Hkv, ps, RANK) if proxy == "loki" else None,
             proj_basis=torch.linalg.qr(torch.randn(Hkv, d, RANK, generator=g))[0].contiguous() if proxy == "loki" else None)
    return c, max(max(lens), 1)


def _decoder(dtype, d, Hq, Hkv, ps, batch, max_ctx, proxy, **kw):
    return SparseDecoder(num_q_heads=Hq, num_kv_heads=Hkv, head_dim=d, dtype=DT[dtype], page_size=ps, max_batch=batch,
                         max_ctx=max_ctx, proxy=proxy, proxy_rank={"exact": 0, "sparq": 16, "loki": RANK}[proxy], **kw)


def _cuda(c):
    """Device copies; views of one wide tensor stay views of one."""
    out = {}
    for key, x in c.items():
        if not isinstance(x, torch.Tensor):
            out[key] = x
        elif x.is_contiguous():
            out[key] = x.cuda()
        else:
            y = torch.empty_strided(x.shape, x.stride(), dtype=x.dtype, device="cuda")
            out[key] = y.copy_(x)
    return out


def _slots(c, new, ps):
    """(token row, sequence, position, page, slot) of every appended token."""
    res, t = [], 0
    for b, n in enumerate(new):
        for i in range(n):
            p = int(c["seq_lens"][b]) - n + i
            res.append((t, b, p, int(c["page_table"][b, p // ps]), p % ps))
            t += 1
    return res


def _tol(ref, mag, dtype):
    # the rotation's bound (tests/test_rotary.py) and the rounding of the stored type
    return 2**-21 * mag + (2**-8 * ref.abs() if dtype == "bf16" else 0)


def _verify(c, x, q_out, new, ps, rope, freq, amp, dtype, proxy):
    slots = _slots(c, new, ps)
    t, _, pos, page, slot = (torch.tensor(v, dtype=torch.int64) for v in zip(*slots))

    def turned(rows):
        return rotate64(rows, pos, rope["rot_dim"], rope["layout"], freq, amp) if rope else rows.double()

    key = turned(c["k"][t])
    kmag = c["k"][t].double().abs().amax(-1, keepdim=True) * 2 * amp if rope else torch.zeros(1)
    got = x["k_cache"].cpu()
    assert ((got[page, :, slot].double() - key).abs() <= _tol(key, kmag, dtype if rope else "f32")).all()
    assert torch.equal(x["v_cache"].cpu()[page, :, slot], c["v"][t])
    # everything else is as it was
    for name in ("k_cache", "v_cache"):
        rest = x[name].cpu().clone()
        rest[page, :, slot] = c[name][page, :, slot]
        assert torch.equal(rest, c[name]), name
    stored = got[page, :, slot]
    if proxy == "sparq":
        kt = x["k_t_cache"].cpu()
        assert torch.equal(kt[page, :, :, slot], stored)
        kt[page, :, :, slot] = c["k_t_cache"][page, :, :, slot]
        assert torch.equal(kt, c["k_t_cache"])
    if proxy == "loki":
        kp = x["k_proj_cache"].cpu()
        b = c["proj_basis"].double()
        ref = torch.einsum("thd,hdr->thr", stored.double(), b)
        mag = torch.einsum("thd,hdr->thr", stored.double().abs(), b.abs())
        tol = stored.shape[-1] * 2**-24 * mag + (2**-8 * ref.abs() if dtype == "bf16" else 0)
        assert ((kp[page, :, slot].double() - ref).abs() <= tol).all()
        kp[page, :, slot] = c["k_proj_cache"][page, :, slot]
        assert torch.equal(kp, c["k_proj_cache"])
    if q_out is not None:
        ref = turned(c["q"][t])
        mag = c["q"][t].double().abs().amax(-1, keepdim=True) * 2 * amp if rope else torch.zeros(1)
        assert ((q_out.cpu()[t].double() - ref).abs() <= _tol(ref, mag, dtype if rope else "f32")).all()


ROPES = [None, dict(rot_dim=64, layout="half"), dict(rot_dim=32, layout="interleaved"), dict(rot_dim=10, layout="half")]


def _run(*, dtype="bf16", d=64, Hq=8, Hkv=2, ps=16, new, before, proxy="exact", rope=1, seed=0, wide=False, pad=0,
         with_q=True, cu=True, kv_location="device", max_batch=None):
    c, max_ctx = _case(dtype=dtype, d=d, Hq=Hq, Hkv=Hkv, ps=ps, new=new, before=before, proxy=proxy, seed=seed,
                       wide=wide, pad=pad)
    rope = ROPES[rope]
    rotary = Rotary(head_dim=d, **rope, scaling="yarn", factor=4.0, original_ctx=64) if rope else None
    freq = frequencies(rope["rot_dim"], scaling="yarn", factor=4.0, original_ctx=64) if rope else None
    amp = amplitude("yarn", 4.0) if rope else 1.0
    dec = _decoder(dtype, d, Hq, Hkv, ps, max_batch or len(new), max_ctx, proxy, kv_location=kv_location)
    x = _cuda(c)
    if kv_location == "host":
        x["k_cache"], x["v_cache"] = c["k_cache"].clone().pin_memory(), c["v_cache"].clone().pin_memory()
    q_out = torch.full((len(x["q"]), Hq, d), 7.0, dtype=DT[dtype], device="cuda") if with_q else None
    res = dec.append(x["k"], x["v"], x["k_cache"], x["v_cache"], x["page_table"], x["seq_lens"], x["num_pages"],
                     cu_tokens=x["cu_tokens"] if cu else None, rotary=rotary, q=x["q"] if with_q else None,
                     q_out=q_out, k_t_cache=x["k_t_cache"], k_proj_cache=x["k_proj_cache"],
                     proj_basis=x["proj_basis"])
    torch.cuda.synchronize()
    assert res is q_out
    assert dec.last_error() == 0
    _verify(c, x, q_out, new, ps, rope, freq, amp, dtype, proxy)
    if with_q:
        assert (q_out[sum(new):] == 7).all()       # rows behind the last sequence
    dec.close()


@pytest.mark.gpu
@pytest.mark.parametrize("proxy", ["exact", "sparq", "loki"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,Hq,Hkv", [(64, 8, 2), (128, 4, 4), (128, 8, 1)])
@pytest.mark.parametrize("rope", range(4))
def test_append_ragged(proxy, dtype, d, Hq, Hkv, rope):
    # empty sequences, one token, pages that end inside, a start in the middle of a page, more than a tile
    _run(dtype=dtype, d=d, Hq=Hq, Hkv=Hkv, new=[5, 0, 1, 130, 16], before=[0, 40, 31, 7, 16], proxy=proxy, rope=rope,
         wide=rope % 2 == 1, pad=3)


@pytest.mark.gpu
@pytest.mark.parametrize("proxy", ["exact", "sparq", "loki"])
@pytest.mark.parametrize("batch", [1, 2, 67])
def test_append_one_token_each(proxy, batch):
    before = [(37 * b) % 200 for b in range(batch)]
    _run(d=128, Hq=32, Hkv=8, new=[1] * batch, before=before, proxy=proxy, cu=False)
    _run(d=128, Hq=32, Hkv=8, new=[1] * batch, before=before, proxy=proxy, cu=True, with_q=False)


@pytest.mark.gpu
@pytest.mark.parametrize("ps", [16, 48, 4096])
@pytest.mark.parametrize("proxy", ["exact", "sparq", "loki"])
def test_append_page_sizes_and_long_prompts(ps, proxy):
    _run(d=128, Hq=8, Hkv=4, ps=ps, new=[1000, 2, 901], before=[3, 1500, 0], proxy=proxy, wide=True)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_append_into_host_caches(dtype):
    _run(dtype=dtype, new=[20, 1], before=[5, 9], kv_location="host")


@pytest.mark.gpu
def test_append_unaligned_rows_and_in_place_queries():
    c, max_ctx = _case(dtype="bf16", d=64, Hq=8, Hkv=2, ps=16, new=[9, 4], before=[2, 30], proxy="exact")
    rotary = Rotary(head_dim=64)
    res = []
    for odd in (False, True):
        dec = _decoder("bf16", 64, 8, 2, 16, 2, max_ctx, "exact")
        x = _cuda(c)
        if odd:      # one element behind a 16-byte boundary
            for key in ("k", "v", "q"):
                flat = torch.zeros(x[key].numel() + 1, dtype=torch.bfloat16, device="cuda")
                flat[1:] = x[key].reshape(-1)
                x[key] = flat[1:].view(x[key].shape)
        out = dec.append(x["k"], x["v"], x["k_cache"], x["v_cache"], x["page_table"], x["seq_lens"], x["num_pages"],
                         cu_tokens=x["cu_tokens"], rotary=rotary, q=x["q"], q_out=x["q"] if odd else None)
        res.append([t.cpu() for t in (out, x["k_cache"], x["v_cache"])])
        assert dec.last_error() == 0
    assert all(torch.equal(a, b) for a, b in zip(*res))


@pytest.mark.gpu
def test_append_skips_and_reports_what_is_out_of_range():
    c, max_ctx = _case(dtype="bf16", d=64, Hq=8, Hkv=2, ps=16, new=[20, 3, 4, 2], before=[0, 10, 0, 5], proxy="exact")
    dec = _decoder("bf16", 64, 8, 2, 16, 4, max_ctx, "exact")
    rotary = Rotary(head_dim=64)

    def call(**kw):
        x = _cuda(dict(c, **kw))
        dec.append(x["k"], x["v"], x["k_cache"], x["v_cache"], x["page_table"], x["seq_lens"], x["num_pages"],
                   cu_tokens=x["cu_tokens"], rotary=rotary)
        err = dec.last_error()
        return x["v_cache"].cpu(), err

    good, err = call()
    assert err == 0
    # the second page of sequence 0 is out of range: its tokens 16..19 alone are missing
    for bad in (-1, c["num_pages"]):
        table = c["page_table"].clone()
        page = int(table[0, 1])
        table[0, 1] = bad
        got, err = call(page_table=table)
        assert err == _abi.VATTN_DEV_BAD_PAGE
        want = good.clone()
        want[page] = c["v_cache"][page]
        assert torch.equal(got, want)
    # a length below the new tokens, and one above max_ctx: that sequence is skipped
    for bad in (2, max_ctx + 1, -5):
        lens = c["seq_lens"].clone()
        lens[1] = bad
        got, err = call(seq_lens=lens)
        assert err == _abi.VATTN_DEV_BAD_SEQLEN
        page = int(c["page_table"][1, 0])
        want = good.clone()
        want[page] = c["v_cache"][page]
        assert torch.equal(got, want)
    # token bounds that descend or leave the rows: the sequences they concern are skipped
    cu = c["cu_tokens"].clone()
    cu[-1] = 99
    got, err = call(cu_tokens=cu)
    assert err == _abi.VATTN_DEV_BAD_SEQLEN
    page = int(c["page_table"][3, 0])
    want = good.clone()
    want[page] = c["v_cache"][page]
    assert torch.equal(got, want)
    dec.close()


@pytest.mark.gpu
def test_append_decode_form_skips_empty_sequences():
    c, max_ctx = _case(dtype="bf16", d=64, Hq=8, Hkv=2, ps=16, new=[1, 1, 1], before=[4, 0, 20], proxy="exact")
    dec = _decoder("bf16", 64, 8, 2, 16, 3, max_ctx, "exact")
    x = _cuda(c)
    x["seq_lens"][1] = 0
    out = torch.full((3, 8, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    dec.append(x["k"], x["v"], x["k_cache"], x["v_cache"], x["page_table"], x["seq_lens"], x["num_pages"],
               q=x["q"], q_out=out)
    assert dec.last_error() == 0
    assert (out[1] == 7).all() and torch.equal(out[[0, 2]], x["q"][[0, 2]])
    page = int(c["page_table"][1, 0])
    assert torch.equal(x["k_cache"][page].cpu(), c["k_cache"][page])
    # lengths out of range are reported
    x["seq_lens"][1] = -1
    dec.append(x["k"], x["v"], x["k_cache"], x["v_cache"], x["page_table"], x["seq_lens"], x["num_pages"])
    assert dec.last_error() == _abi.VATTN_DEV_BAD_SEQLEN
    dec.close()


@pytest.mark.gpu
def test_append_far_offsets_in_a_large_cache():
    # cache rows behind 2^32 elements: 2 GiB-crossing byte offsets in both caches
    ps, Hkv, d = 65536, 2, 64
    pages = 520                                     # 520 * 2 * 65536 * 64 = 4.36e9 elements
    dec = _decoder("bf16", d, 2, Hkv, ps, 1, ps, "exact")
    k_cache = torch.zeros((pages, Hkv, ps, d), dtype=torch.bfloat16, device="cuda")
    v_cache = torch.zeros((pages, Hkv, ps, d), dtype=torch.bfloat16, device="cuda")
    k, v = (torch.randn(3, Hkv, d, device="cuda").bfloat16() for _ in range(2))
    i32 = dict(dtype=torch.int32, device="cuda")
    dec.append(k, v, k_cache, v_cache, torch.tensor([[pages - 1]], **i32), torch.tensor([ps], **i32), pages,
               cu_tokens=torch.tensor([0, 3], **i32))
    assert dec.last_error() == 0
    assert torch.equal(k_cache[pages - 1, :, ps - 3:].transpose(0, 1), k)
    assert torch.equal(v_cache[pages - 1, :, ps - 3:].transpose(0, 1), v)
    assert not v_cache[:pages - 1].any() and not v_cache[pages - 1, :, :ps - 3].any()
    dec.close()


@pytest.mark.gpu
def test_append_captured_with_growing_lengths():
    c, max_ctx = _case(dtype="bf16", d=64, Hq=8, Hkv=2, ps=16, new=[1, 1], before=[40, 25], proxy="exact")
    dec = _decoder("bf16", 64, 8, 2, 16, 2, max_ctx, "exact")
    x = _cuda(c)
    rotary = Rotary(head_dim=64)
    out = torch.zeros_like(x["q"])

    def step():
        dec.append(x["k"], x["v"], x["k_cache"], x["v_cache"], x["page_table"], x["seq_lens"], x["num_pages"],
                   rotary=rotary, q=x["q"], q_out=out)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    x["seq_lens"] -= 9
    for _ in range(9):
        x["seq_lens"] += 1
        x["k"] += 1
        graph.replay()
    ref = _cuda(c)
    ref["seq_lens"] -= 9
    for _ in range(9):
        ref["seq_lens"] += 1
        ref["k"] += 1
        want = dec.append(ref["k"], ref["v"], ref["k_cache"], ref["v_cache"], ref["page_table"], ref["seq_lens"],
                          ref["num_pages"], rotary=rotary, q=ref["q"])
    assert dec.last_error() == 0
    assert torch.equal(out, want) and torch.equal(x["k_cache"], ref["k_cache"])
    assert torch.equal(x["v_cache"], ref["v_cache"])
    dec.close()


@pytest.mark.gpu
def test_append_calls_of_one_context_may_overlap():
    c, max_ctx = _case(dtype="bf16", d=128, Hq=8, Hkv=2, ps=16, new=[400, 300], before=[3, 60], proxy="loki")
    dec = _decoder("bf16", 128, 8, 2, 16, 2, max_ctx, "loki")
    rotary = Rotary(head_dim=128)

    def call(x, stream=None):
        dec.append(x["k"], x["v"], x["k_cache"], x["v_cache"], x["page_table"], x["seq_lens"], x["num_pages"],
                   cu_tokens=x["cu_tokens"], rotary=rotary, q=x["q"], q_out=x["q_out"],
                   k_proj_cache=x["k_proj_cache"], proj_basis=x["proj_basis"], stream=stream)

    xs = [_cuda(c) for _ in range(3)]
    for x in xs:
        x["q_out"] = torch.empty_like(x["q"])
    call(xs[0])
    torch.cuda.synchronize()
    for x in xs[1:]:
        call(x, torch.cuda.Stream())
    torch.cuda.synchronize()
    assert dec.last_error() == 0
    for x in xs[1:]:
        assert all(torch.equal(x[k], xs[0][k]) for k in ("k_cache", "v_cache", "k_proj_cache", "q_out"))
    dec.close()


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_append_basis_at_any_float(d):
    c, max_ctx = _case(dtype="bf16", d=d, Hq=4, Hkv=2, ps=16, new=[70, 0, 33], before=[5, 9, 0], proxy="loki")
    dec = _decoder("bf16", d, 4, 2, 16, 3, max_ctx, "loki")
    got = []
    for shift in (0, 1):
        x = _cuda(c)
        flat = torch.empty(x["proj_basis"].numel() + 1, device="cuda")
        basis = flat[shift:shift + x["proj_basis"].numel()].view_as(x["proj_basis"])
        basis.copy_(x["proj_basis"])
        assert basis.data_ptr() % 16 == 4 * shift
        dec.append(x["k"], x["v"], x["k_cache"], x["v_cache"], x["page_table"], x["seq_lens"], x["num_pages"],
                   cu_tokens=x["cu_tokens"], k_proj_cache=x["k_proj_cache"], proj_basis=basis)
        torch.cuda.synchronize()
        got.append(x)
    # the same products in the same order, whatever the access width
    for k in ("k_cache", "v_cache", "k_proj_cache"):
        assert torch.equal(got[0][k], got[1][k])
    dec.close()


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_append_projects_with_the_whole_fp32_basis(d):
    # keys of one +1 and one -1: the projected key is the difference of two basis entries, which agree but for
    # their last 12 bits. At most six products (three bf16 terms of each entry, below 2) are not zero, and an
    # fp32 accumulator loses up to 2^-23 of its magnitude with each; then the result is rounded to bf16. The
    # stored rotated key is the key itself (no rotation).
    c, max_ctx = _case(dtype="bf16", d=d, Hq=4, Hkv=2, ps=16, new=[70, 0, 33], before=[5, 9, 0], proxy="loki")
    g = torch.Generator().manual_seed(3)
    T = len(c["k"])
    at = torch.stack([torch.randperm(d, generator=g)[:2] for _ in range(2 * T)]).view(T, 2, 2)
    c["k"] = torch.zeros(T, 2, d).scatter_(2, at, torch.tensor([1.0, -1.0]).expand(T, 2, 2)).bfloat16()
    c["proj_basis"] = 1 + torch.rand(2, 1, RANK, generator=g) / 2 + 2**-12 * torch.rand(2, d, RANK, generator=g)
    dec = _decoder("bf16", d, 4, 2, 16, 3, max_ctx, "loki")
    x = _cuda(c)
    dec.append(x["k"], x["v"], x["k_cache"], x["v_cache"], x["page_table"], x["seq_lens"], x["num_pages"],
               cu_tokens=x["cu_tokens"], k_proj_cache=x["k_proj_cache"], proj_basis=x["proj_basis"])
    assert dec.last_error() == 0
    t, _, _, page, slot = (torch.tensor(v, dtype=torch.int64) for v in zip(*_slots(c, [70, 0, 33], 16)))
    ref = torch.einsum("thd,hdr->thr", c["k"][t].double(), c["proj_basis"].double())
    err = (x["k_proj_cache"].cpu()[page, :, slot].double() - ref).abs() - 2**-8 * ref.abs()
    assert float(err.max()) <= 6 * 2**-23 * 2, float(err.max())
    dec.close()


@pytest.mark.gpu
@pytest.mark.parametrize("length", [-2**31, -2**31 + 1, -2**31 + 3, 2**31 - 1])
def test_append_skips_and_reports_lengths_at_the_ends_of_int32(length):
    c, max_ctx = _case(dtype="bf16", d=64, Hq=8, Hkv=2, ps=16, new=[20, 3, 4, 2], before=[0, 10, 0, 5], proxy="exact")
    dec = _decoder("bf16", 64, 8, 2, 16, 4, max_ctx, "exact")
    lens = c["seq_lens"].clone()
    lens[1] = length
    for rows, cu in ((slice(None), c["cu_tokens"].cuda()), (slice(4), None)):   # ragged, and one token each
        got = []
        for seq_lens in (c["seq_lens"], lens):
            x = _cuda(dict(c, seq_lens=seq_lens))
            dec.append(x["k"][rows], x["v"][rows], x["k_cache"], x["v_cache"], x["page_table"], x["seq_lens"],
                       x["num_pages"], cu_tokens=cu)
            assert dec.last_error() == (0 if seq_lens is c["seq_lens"] else _abi.VATTN_DEV_BAD_SEQLEN)
            got.append([x["k_cache"].cpu(), x["v_cache"].cpu()])
        page = int(c["page_table"][1, 0])
        for name, good, bad in zip(("k_cache", "v_cache"), *got):
            good[page] = c[name][page]
            assert torch.equal(bad, good)
    dec.close()


@pytest.mark.gpu
@pytest.mark.parametrize("proxy", ["exact", "sparq"])
def test_append_bounds_that_descend(proxy):
    # sequence 1's bounds descend: it is skipped, and the rows that sequences 0 and 2 both claim are sequence 0's
    new = [30, 5, 20, 7]
    c, max_ctx = _case(dtype="bf16", d=64, Hq=8, Hkv=2, ps=16, new=new, before=[3, 10, 30, 0], proxy=proxy, pad=5)
    dec = _decoder("bf16", 64, 8, 2, 16, 4, max_ctx, proxy)
    cu = torch.tensor([0, 30, 22, 42, 49], dtype=torch.int32)
    want = {k: c[k].clone() for k in ("k_cache", "v_cache")}
    q_want = torch.full_like(c["q"], 7.0)
    for b, rows in ((0, range(30)), (2, range(30, 42)), (3, range(42, 49))):
        for t in rows:
            p = int(c["seq_lens"][b]) - int(cu[b + 1]) + t
            page, slot = int(c["page_table"][b, p // 16]), p % 16
            want["k_cache"][page, :, slot], want["v_cache"][page, :, slot] = c["k"][t], c["v"][t]
            q_want[t] = c["q"][t]
    for _ in range(5):
        x = _cuda(c)
        out = torch.full_like(x["q"], 7.0)
        dec.append(x["k"], x["v"], x["k_cache"], x["v_cache"], x["page_table"], x["seq_lens"], x["num_pages"],
                   cu_tokens=cu.cuda(), q=x["q"], q_out=out, k_t_cache=x["k_t_cache"])
        assert dec.last_error() == _abi.VATTN_DEV_BAD_SEQLEN
        assert torch.equal(x["k_cache"].cpu(), want["k_cache"]) and torch.equal(x["v_cache"].cpu(), want["v_cache"])
        assert torch.equal(out.cpu(), q_want)
    dec.close()


@pytest.mark.gpu
def test_append_reports_bad_lengths_of_sequences_without_new_tokens():
    c, max_ctx = _case(dtype="bf16", d=64, Hq=8, Hkv=2, ps=16, new=[70, 0, 5], before=[0, 10, 3], proxy="exact")
    dec = _decoder("bf16", 64, 8, 2, 16, 3, max_ctx, "exact")
    got = []
    for length in (10, 0, -1, max_ctx + 1):
        lens = c["seq_lens"].clone()
        lens[1] = length
        x = _cuda(dict(c, seq_lens=lens))
        dec.append(x["k"], x["v"], x["k_cache"], x["v_cache"], x["page_table"], x["seq_lens"], x["num_pages"],
                   cu_tokens=x["cu_tokens"])
        assert dec.last_error() == (0 if 0 <= length <= max_ctx else _abi.VATTN_DEV_BAD_SEQLEN), length
        got.append(x)
    for x in got[1:]:
        assert torch.equal(x["k_cache"], got[0]["k_cache"]) and torch.equal(x["v_cache"], got[0]["v_cache"])
    dec.close()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_append_refuses_pointers_between_elements(dtype):
    c, max_ctx = _case(dtype=dtype, d=64, Hq=8, Hkv=2, ps=16, new=[3, 2], before=[2, 30], proxy="loki")
    dec = _decoder(dtype, 64, 8, 2, 16, 2, max_ctx, "loki")
    x = _cuda(c)
    out = torch.zeros_like(x["q"])

    def rc(table=0, lens=0, **off):
        a = dict(k=x["k"], v=x["v"], q=x["q"], q_out=out, k_cache=x["k_cache"], v_cache=x["v_cache"],
                 k_proj_cache=x["k_proj_cache"], proj_basis=x["proj_basis"], cu_tokens=x["cu_tokens"])
        a = {k: t.data_ptr() + off.get(k, 0) for k, t in a.items()}
        p = _abi.vattn_append_params(tokens=5, num_pages=x["num_pages"], k_stride=128, v_stride=128, q_stride=512, **a)
        return _abi.vattn_append(dec.ctx, p, x["page_table"].data_ptr() + table, x["seq_lens"].data_ptr() + lens, 2,
                                 check=False)

    for name in ("k", "v", "q", "q_out"):
        for off in ((1,) if dtype == "bf16" else (1, 2, 3)):
            assert rc(**{name: off}) == _abi.VATTN_EINVAL, name
    for name in ("table", "lens", "cu_tokens", "proj_basis"):
        for off in (1, 2, 3):
            assert rc(**{name: off}) == _abi.VATTN_EINVAL, name
    for name in ("k_cache", "v_cache", "k_proj_cache"):
        assert rc(**{name: 8}) == _abi.VATTN_EINVAL, name
    assert torch.equal(x["k_cache"].cpu(), c["k_cache"]) and not out.any()
    assert rc() == _abi.VATTN_OK and dec.last_error() == 0
    dec.close()


@pytest.mark.gpu
def test_append_one_token_of_a_wide_row_in_place():
    c, max_ctx = _case(dtype="bf16", d=64, Hq=8, Hkv=2, ps=16, new=[1], before=[20], proxy="exact", wide=True)
    dec = _decoder("bf16", 64, 8, 2, 16, 1, max_ctx, "exact")
    rotary = Rotary(head_dim=64)
    x = _cuda(c)
    want = dec.append(x["k"], x["v"], x["k_cache"], x["v_cache"], x["page_table"], x["seq_lens"], x["num_pages"],
                      rotary=rotary, q=x["q"])
    y = _cuda(c)
    wide = torch.cat([c["q"], c["k"], c["v"], c["v"][:, :1]], 1).cuda()
    keep = wide.clone()
    q = wide[:, :8]
    assert dec.append(wide[:, 8:10], wide[:, 10:12], y["k_cache"], y["v_cache"], y["page_table"], y["seq_lens"],
                      y["num_pages"], rotary=rotary, q=q, q_out=q) is q
    assert dec.last_error() == 0
    assert torch.equal(q, want) and torch.equal(wide[:, 8:], keep[:, 8:])
    assert torch.equal(y["k_cache"], x["k_cache"]) and torch.equal(y["v_cache"], x["v_cache"])
    dec.close()
