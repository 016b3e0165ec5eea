"""vattn_shared_dense_decode against 64-bit attention over every sequence's own pages."""
import math

import pytest
import torch

from tests.serving import dense64, frequencies, rotate64, shared_batch
from tests.test_append import _fake
from verified_sparse_attention_b200 import _abi
from verified_sparse_attention_b200.decoder import SparseDecoder
from verified_sparse_attention_b200.rotary import Rotary

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------ refusals of the wrapper (CPU)
def _args(**kw):
    bf, i32 = torch.bfloat16, torch.int32
    a = dict(q=torch.zeros(3, 8, 64, dtype=bf), k_cache=torch.zeros(5, 2, 16, 64, dtype=bf),
             v_cache=torch.zeros(5, 2, 16, 64, dtype=bf), page_table=torch.zeros(3, 7, dtype=i32),
             seq_lens=torch.ones(3, dtype=i32), num_pages=5, group_start=torch.tensor([0, 3], dtype=i32),
             prefix_lens=torch.zeros(1, dtype=i32))
    a.update(kw)
    return a


@pytest.mark.parametrize("bad", [
    dict(q=torch.zeros(3, 8, 64)), dict(q=torch.zeros(2, 8, 64, dtype=torch.bfloat16)),
    dict(q=torch.zeros(8, 3, 64, dtype=torch.bfloat16).transpose(0, 1)),
    dict(group_start=torch.tensor([0, 1, 3], dtype=torch.int32)), dict(group_start=torch.tensor([0, 3])),
    dict(prefix_lens=torch.zeros(1)), dict(out=torch.zeros(3, 8, 64, dtype=torch.bfloat16)),
    dict(out=torch.zeros(3, 8, 32)), dict(num_pages=6), dict(k_cache=torch.zeros(5, 2, 16, 64))])
def test_shared_wrapper_refusals(bad):
    with pytest.raises(ValueError):
        _fake().shared_dense(**_args(**bad))


def test_shared_needs_a_context():
    with pytest.raises(_abi.VattnError):
        _fake().shared_dense(**_args())


# ------------------------------------------------------------ on the GPU
def _tol(x, d):
    """|out - exact| for one output, over max |v|.

    A score is a sum of d exact products in fp32: d 2^-24 sum |q k| / sqrt(d) at most, sum |q k| under
    3 d for these normal inputs; its scaling and the difference to the maximum add 2^-23 of |s| <= 16. The
    weight exp2 adds 2^-21, and 2^-17 where it is split into two bf16 terms; the sums of weights and products
    at most 2^-16 in all. Numerator and denominator: twice that."""
    score = d * 2**-24 * 3 * d / math.sqrt(d) + 2**-19
    return 2 * (score + 2**-21 + 2**-17 + 2**-16) * float(torch.nan_to_num(x["v_cache"].float()).abs().max())


def _decoder(x, dtype, ps, max_batch=None, **kw):
    B, Hq, d = x["q"].shape
    return SparseDecoder(num_q_heads=Hq, num_kv_heads=x["k_cache"].shape[1], head_dim=d, dtype=DT[dtype], page_size=ps,
                         max_batch=max_batch or max(B, len(x["prefix_lens"])), max_ctx=x["max_ctx"], **kw)


def _cuda(x):
    return {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in x.items()}


def _call(dec, x, **kw):
    return dec.shared_dense(x["q"], x["k_cache"], x["v_cache"], x["page_table"], x["seq_lens"], x["num_pages"],
                            x["group_start"], x["prefix_lens"], **kw)


def _run(sizes, prefixes, own, *, dtype="bf16", d=128, Hq=8, Hkv=2, ps=16, seed=0, kv_location="device"):
    x = shared_batch(sizes, prefixes, own, Hq=Hq, Hkv=Hkv, d=d, ps=ps, dtype=DT[dtype], seed=seed)
    dec = _decoder(x, dtype, ps, kv_location=kv_location)
    y = _cuda(x)
    if kv_location == "host":
        y["k_cache"], y["v_cache"] = x["k_cache"].pin_memory(), x["v_cache"].pin_memory()
    got = _call(dec, y, out=torch.full((len(x["q"]), Hq, d), float("nan"), device="cuda")).cpu().double()
    assert dec.last_error() == 0
    ref = dense64(x["q"], x["k_cache"], x["v_cache"], x["page_table"], x["seq_lens"])
    assert (got[x["seq_lens"] == 0] == 0).all()
    err = float((got - ref).abs().max())
    assert err <= _tol(x, d), err
    dec.close()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(2, 2), (4, 2), (4, 1), (16, 2)])
@pytest.mark.parametrize("prefix", [1, 15, 16, 127, 128, 129, 1000])
def test_shared_one_group(dtype, d, Hq, Hkv, prefix):
    _run([5], [prefix], [0, 1, 17, 70, 3], dtype=dtype, d=d, Hq=Hq, Hkv=Hkv)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("ps", [16, 32, 48, 64, 128, 2048])
def test_shared_groups_of_every_kind(dtype, ps):
    # alone, two, many; no prefix; sequences short of the prefix, at its end, empty; a group all empty
    sizes = [1, 2, 9, 3, 2, 1, 4]
    prefixes = [300, 257, 700, 0, 50, 0, 513]
    own = [5, 40, 0, 1, 2, 3, -699, 0, 31, -700, -100, 64, 10, 0, 200, -50, -50, 129, 8, -1, 20, 0]
    _run(sizes, prefixes, own, dtype=dtype, ps=ps)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,Hq,Hkv", [(33, 8, 2), (40, 8, 1), (64, 8, 2), (70, 8, 2), (129, 8, 1), (150, 2, 2)])
def test_shared_many_rows(dtype, B, Hq, Hkv):
    # rows that fill one tile of 128 or 256, or pass it
    _run([B], [400], [(7 * b) % 50 for b in range(B)], dtype=dtype, Hq=Hq, Hkv=Hkv, d=64)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("groups,size,prefix", [(17, 2, 40), (40, 3, 150), (1, 400, 200), (1100, 1, 0), (700, 2, 33)])
def test_shared_many_groups_and_sequences(dtype, groups, size, prefix):
    # more groups or sequences than the kernels keep in shared memory
    B = groups * size
    _run([size] * groups, [max(prefix - g % 7, 0) for g in range(groups)], [(5 * b) % 23 for b in range(B)], dtype=dtype,
         d=64, Hq=2, Hkv=1)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_shared_empty_groups(dtype):
    _run([0, 3, 0, 0, 2, 0], [40, 100, 0, 7, 64, 1], [1, 5, 0, 20, 33], dtype=dtype, d=64)


@pytest.mark.gpu
@pytest.mark.parametrize("B,heads,prefix", [(3, 16, 100000), (140, 16, 40000), (2, 1, 130001)])
def test_shared_prefix_of_many_tiles(B, heads, prefix):
    # more key tiles in a row than one accumulator takes, one and two query tiles
    g = torch.Generator(device="cuda").manual_seed(5)
    d, ps = 64, 1024
    whole, own = prefix // ps, 3 + prefix % ps
    pages = whole + B
    k, v = (torch.randn(pages, heads, ps * 2, d, generator=g, device="cuda").bfloat16()[:, :, :ps].contiguous()
            for _ in range(2))
    i32 = dict(dtype=torch.int32, device="cuda")
    table = torch.cat([torch.arange(whole, **i32).expand(B, whole), whole + torch.arange(B, **i32)[:, None]], 1).contiguous()
    # the page in which the prefix ends holds the same rows in every sequence
    for c in (k, v):
        c[whole + 1:, :, :prefix % ps] = c[whole, :, :prefix % ps].clone()
    x = dict(q=torch.randn(B, heads, d, generator=g, device="cuda").bfloat16(), k_cache=k, v_cache=v, page_table=table,
             seq_lens=torch.full((B,), whole * ps + own, **i32), group_start=torch.tensor([0, B], **i32),
             prefix_lens=torch.tensor([prefix], **i32), num_pages=pages, max_ctx=(whole + 1) * ps)
    # scores that rise along the prefix move the maximum behind the first accumulators
    grow = torch.linspace(0.5, 2.0, whole, device="cuda")[:, None, None, None]
    k[:whole] = (k[:whole].float() * grow).bfloat16()
    dec = _decoder(x, "bf16", ps)
    got = _call(dec, x).double()
    assert dec.last_error() == 0
    ref = dense64(x["q"], k, v, table, x["seq_lens"])
    assert float((got - ref).abs().max()) <= 2 * _tol(x, d)    # keys of twice the size
    dec.close()


@pytest.mark.gpu
def test_shared_long_prefix():
    _run([6, 10], [20001, 9000], [(31 * b) % 300 for b in range(16)], Hq=16, Hkv=4)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_shared_host_caches(dtype):
    _run([3, 2], [200, 77], [1, 20, 0, 5, 40], dtype=dtype, kv_location="host")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_shared_large_scores_and_rising_maxima(dtype):
    # keys that grow along the prefix: every tile raises the maximum, far above the earlier ones
    x = shared_batch([40], [900], [(3 * b) % 40 for b in range(40)], Hq=8, Hkv=2, d=64, ps=16, dtype=DT[dtype], seed=3,
                     garbage=0.0)
    pages = x["page_table"][0, :56].long()
    x["q"] = x["q"].abs()
    grow = torch.linspace(0.0, 4.0, 56)[:, None, None, None]
    x["k_cache"][pages] = (x["k_cache"][pages].float().abs() * grow).to(DT[dtype])
    y = _cuda(x)
    dec = _decoder(x, dtype, 16)
    got = _call(dec, y).cpu().double()
    ref = dense64(x["q"], x["k_cache"], x["v_cache"], x["page_table"], x["seq_lens"])
    # scores up to ~ 4 * 64 * 0.64 / 8 = 20 with partial sums as large: 4 times the products of _tol's bound
    assert float((got - ref).abs().max()) <= 4 * _tol(x, 64)
    assert dec.last_error() == 0
    dec.close()


@pytest.mark.gpu
def test_shared_reports_and_zeroes_what_is_out_of_range():
    x = shared_batch([3, 4], [100, 60], [5, 9, 0, 1, 30, 2, 8], Hq=8, Hkv=2, d=64, ps=16, dtype=torch.bfloat16)
    dec = _decoder(x, "bf16", 16)
    ref = _call(dec, _cuda(x)).cpu()
    assert dec.last_error() == 0

    def call(zero, bit, **kw):
        got = _call(dec, _cuda(dict(x, **kw))).cpu()
        assert dec.last_error() == bit
        rest = [b for b in range(7) if b not in zero]
        assert not got[zero].any()
        # other splits of the work sum in another order
        assert not rest or float((got[rest] - ref[rest]).abs().max()) <= 2 * _tol(x, 64)

    def changed(key, at, value):
        t = x[key].clone()
        t[at] = value
        return {key: t}

    BAD_LEN, BAD_PAGE, BAD_GROUP = _abi.VATTN_DEV_BAD_SEQLEN, _abi.VATTN_DEV_BAD_PAGE, _abi.VATTN_DEV_BAD_GROUP
    call([0, 1, 2], BAD_PAGE, **changed("page_table", (0, 2), x["num_pages"]))  # a prefix page of group 0
    call([4], BAD_PAGE, **changed("page_table", (4, 5), -1))                    # an own page of sequence 4
    call([1], BAD_LEN, **changed("seq_lens", 1, x["max_ctx"] + 1))
    call([1], BAD_LEN, **changed("seq_lens", 1, -1))
    call([3, 4, 5, 6], BAD_GROUP, **changed("prefix_lens", 1, x["max_ctx"] + 1))
    call([3, 4, 5, 6], BAD_GROUP, **changed("prefix_lens", 1, -1))
    every = list(range(7))
    call(every, BAD_GROUP, **changed("group_start", 0, 1))
    call(every, BAD_GROUP, **changed("group_start", 1, 9))
    call(every, BAD_GROUP, **changed("group_start", 2, 6))
    dec.close()


@pytest.mark.gpu
def test_shared_refusals_before_any_launch():
    x = shared_batch([2], [20], [1, 2], Hq=8, Hkv=2, d=64, ps=16, dtype=torch.bfloat16)
    dec = _decoder(x, "bf16", 16)
    y = _cuda(x)
    out = torch.full((2, 8, 64), 5.0, device="cuda")

    def rc(**kw):
        a = dict(q=y["q"], k_cache=y["k_cache"], v_cache=y["v_cache"], page_table=y["page_table"],
                 seq_lens=y["seq_lens"], group_start=y["group_start"], prefix_lens=y["prefix_lens"], groups=1, batch=2,
                 num_pages=x["num_pages"], out=out)
        a.update(kw)
        return _abi.vattn_shared_dense_decode(dec.ctx, *a.values(), check=False)

    for bad in (dict(q=None), dict(k_cache=None), dict(page_table=None), dict(group_start=None),
                dict(prefix_lens=None), dict(out=None), dict(groups=0), dict(groups=-1), dict(batch=-1), dict(batch=3),
                dict(num_pages=0), dict(q=y["q"].data_ptr() + 2), dict(k_cache=y["k_cache"].data_ptr() + 8)):
        assert rc(**bad) == _abi.VATTN_EINVAL, bad
    assert rc(batch=0, groups=0, q=None) == _abi.VATTN_OK
    assert (out == 5).all()
    dec.close()


@pytest.mark.gpu
def test_shared_captured_on_another_stream_with_a_padded_batch():
    x = shared_batch([6, 5], [300, 130], [(5 * b) % 20 for b in range(11)], Hq=8, Hkv=2, d=64, ps=16,
                     dtype=torch.bfloat16)
    dec = _decoder(x, "bf16", 16)
    y = _cuda(x)
    out = torch.zeros(11, 8, 64, device="cuda")
    graph = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=s):
        _call(dec, y, out=out)
    # a step later: other lengths, two slots empty, the second group larger
    lens = x["seq_lens"].clone()
    lens[3] = 0
    lens[10] = 0
    y["seq_lens"].copy_(lens)
    graph.replay()
    got = out.cpu().double()
    ref = dense64(x["q"], x["k_cache"], x["v_cache"], x["page_table"], lens)
    assert float((got - ref).abs().max()) <= _tol(x, 64)
    assert dec.last_error() == 0
    dec.close()


@pytest.mark.gpu
def test_shared_equals_dense_and_is_reproducible():
    x = shared_batch([20], [2000], [(11 * b) % 90 for b in range(20)], Hq=16, Hkv=4, d=128, ps=16, dtype=torch.bfloat16,
                     garbage=0.0)
    dec = _decoder(x, "bf16", 16)
    y = _cuda(x)
    a, b = _call(dec, y), _call(dec, y)
    assert torch.equal(a, b)
    dense = dec.dense(y["q"], y["k_cache"], y["v_cache"], y["page_table"], y["seq_lens"], y["num_pages"])
    assert float((a - dense).abs().max()) <= 2 * _tol(x, 128)
    dec.close()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_shared_two_contexts_on_two_streams(dtype):
    xs = [shared_batch([9, 6], [700 + 50 * i, 90], [(5 * b + i) % 30 for b in range(15)], Hq=8, Hkv=2, d=64, ps=16,
                       dtype=DT[dtype], seed=i) for i in range(2)]
    decs = [_decoder(x, dtype, 16) for x in xs]
    ys = [_cuda(x) for x in xs]
    ref = [_call(d, y).clone() for d, y in zip(decs, ys)]
    outs = [torch.zeros_like(r) for r in ref]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for d, y, o, s in zip(decs, ys, outs, streams):
            _call(d, y, out=o, stream=s)
    torch.cuda.synchronize()
    for d, o, r in zip(decs, outs, ref):
        assert torch.equal(o, r) and d.last_error() == 0
        d.close()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,kv_location", [("bf16", "device"), ("f32", "device"), ("f32", "host")])
def test_shared_output_at_any_float(dtype, kv_location):
    x = shared_batch([3, 2], [200, 77], [1, 20, 0, 5, 40], Hq=8, Hkv=2, d=64, ps=16, dtype=DT[dtype])
    dec = _decoder(x, dtype, 16, kv_location=kv_location)
    y = _cuda(x)
    if kv_location == "host":
        y["k_cache"], y["v_cache"] = x["k_cache"].pin_memory(), x["v_cache"].pin_memory()
    ref = _call(dec, y)
    flat = torch.full((ref.numel() + 4,), 3.0, device="cuda")
    for shift in range(4):
        flat.fill_(3.0)
        _call(dec, y, out=flat[shift:shift + ref.numel()].view_as(ref))
        assert torch.equal(flat[shift:shift + ref.numel()].view_as(ref), ref)
        assert (flat[:shift] == 3).all() and (flat[shift + ref.numel():] == 3).all()
    assert dec.last_error() == 0
    dec.close()


@pytest.mark.gpu
def test_shared_refuses_pointers_between_elements():
    x = shared_batch([2], [20], [1, 2], Hq=8, Hkv=2, d=64, ps=16, dtype=torch.bfloat16)
    dec = _decoder(x, "bf16", 16)
    y = _cuda(x)
    out = torch.full((2, 8, 64), 5.0, device="cuda")

    def rc(**off):
        a = dict(q=y["q"], k_cache=y["k_cache"], v_cache=y["v_cache"], page_table=y["page_table"],
                 seq_lens=y["seq_lens"], group_start=y["group_start"], prefix_lens=y["prefix_lens"])
        a = [t.data_ptr() + off.get(k, 0) for k, t in a.items()]
        return _abi.vattn_shared_dense_decode(dec.ctx, *a, 1, 2, x["num_pages"], out.data_ptr() + off.get("out", 0),
                                              check=False)

    for name in ("page_table", "seq_lens", "group_start", "prefix_lens", "out"):
        for off in (1, 2, 3):
            assert rc(**{name: off}) == _abi.VATTN_EINVAL, name
    for name in ("q", "k_cache", "v_cache"):
        assert rc(**{name: 4}) == _abi.VATTN_EINVAL, name
    assert (out == 5).all()
    assert rc() == _abi.VATTN_OK and dec.last_error() == 0
    dec.close()


@pytest.mark.gpu
@pytest.mark.parametrize("unlisted", ["invalid", "stale"])
@pytest.mark.parametrize("dtype,ps,kv_location", [("bf16", 16, "device"), ("bf16", 48, "device"), ("bf16", 2048, "device"),
                                                  ("f32", 16, "device"), ("f32", 48, "device"), ("f32", 2048, "device"),
                                                  ("f32", 16, "host"), ("bf16", 48, "host")])
def test_shared_prefix_is_read_through_the_first_sequence(dtype, ps, kv_location, unlisted):
    # one, two, three or all of a group reach the prefix's end, with the first and without it; only the first lists
    # the prefix's pages, and the others' rows of the page that it ends in hold nothing of it
    sizes, prefixes = [3, 2, 4, 3, 1, 6], [100, 57, 200, 64, 30, 90]
    own = [-50, -100, 20, -10, 5, -3, 40, 0, -200, 0, 1, 33, 7, -1, 3, -90, 50, 16, 0]
    x = shared_batch(sizes, prefixes, own, Hq=8, Hkv=2, d=64, ps=ps, dtype=DT[dtype], seed=4)
    ref = dense64(x["q"], x["k_cache"], x["v_cache"], x["page_table"], x["seq_lens"])
    k, v, table = x["k_cache"].clone(), x["v_cache"].clone(), x["page_table"].clone()
    used = torch.zeros(x["num_pages"], dtype=torch.bool)
    used[table[table >= 0].long()] = True
    stale = int((~used).nonzero()[0])                    # a page of garbage
    start = x["group_start"].tolist()
    for g, prefix in enumerate(prefixes):
        for b in range(start[g] + 1, start[g + 1]):
            if int(x["seq_lens"][b]) < prefix:
                continue
            whole, rest = divmod(prefix, ps)
            table[b, :whole] = -1 if unlisted == "invalid" else stale
            if rest and int(x["seq_lens"][b]) == prefix:
                table[b, whole] = -1 if unlisted == "invalid" else stale
            elif rest:
                k[int(table[b, whole]), :, :rest] = float("nan")
                v[int(table[b, whole]), :, :rest] = float("nan")
    dec = _decoder(x, dtype, ps, kv_location=kv_location)
    y = _cuda(dict(x, k_cache=k, v_cache=v, page_table=table))
    if kv_location == "host":
        y["k_cache"], y["v_cache"] = k.pin_memory(), v.pin_memory()
    got = _call(dec, y).cpu().double()
    assert dec.last_error() == 0
    assert float((got - ref).abs().max()) <= _tol(x, 64)
    # a first sequence that lists a bad page: those that read it give zeros and it is reported, the others (short of
    # the prefix) are decoded from their own pages
    for page in (-1, x["num_pages"]):
        bad = y["page_table"].clone()
        bad[start[2], 0] = page                          # group 2: sequences 5 (first, short), 6, 7, 8 (empty)
        got = _call(dec, dict(y, page_table=bad)).cpu().double()
        assert dec.last_error() == _abi.VATTN_DEV_BAD_PAGE
        assert not got[[5, 6, 7, 8]].any()
        rest = [b for b in range(len(own)) if not 5 <= b < 9]
        assert float((got - ref)[rest].abs().max()) <= _tol(x, 64)
    dec.close()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("prefix", [0, 200])
def test_shared_scores_far_below_zero(dtype, prefix):
    # every key has the same score, about -1.6e32 (exact: one product of powers of two): the mean of the values
    x = shared_batch([6], [prefix], [5, 1, 40, 17, 9, 3], Hq=8, Hkv=2, d=64, ps=16, dtype=DT[dtype], seed=6)
    x["q"] = torch.zeros_like(x["q"])
    x["q"][..., 3] = 2.0**60
    k = torch.zeros_like(x["k_cache"])
    k[..., 3] = -2.0**50
    x["k_cache"] = torch.where(x["k_cache"].isnan(), x["k_cache"], k)
    dec = _decoder(x, dtype, 16)
    got = _call(dec, _cuda(x)).cpu().double()
    assert dec.last_error() == 0
    ref = dense64(x["q"], x["k_cache"], x["v_cache"], x["page_table"], x["seq_lens"])
    assert float((got - ref).abs().max()) <= _tol(x, 64)
    dec.close()


# ------------------------------------------------------------ precision
def _row_errors(got, ref):
    """|got - ref| of every row over the row's norm (rows that are not zero)."""
    norm = ref.norm(dim=-1)
    return ((got - ref).norm(dim=-1) / norm)[norm > 0]


# For random values the error of a row is at most the weights' relative error times the row's norm, as the errors of
# different keys do not add up. A weight of the bf16 kernels is two bf16 terms, 2^-8 of 2^-8 off at most (1.5e-5); the
# tensor core's truncation takes up to 7e-6 from every component; fp32 scores, exponentials and sums are a few 1e-6 off.
# A second term left out is 1e-3, a key of 20001 left out 7e-3, a tile of 128 keys in 130000 3e-2.
ROW_TOL = 4e-5


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("sizes,prefixes,ps", [([5], [300], 16), ([3, 8, 1, 6], [1000, 129, 40, 513], 48),
                                               ([40], [700], 128), ([70, 10], [400, 128], 64), ([6, 10], [20001, 9000], 16),
                                               ([2] * 20, [100] * 20, 16)])
def test_shared_rows_are_precise(dtype, d, sizes, prefixes, ps):
    B = sum(sizes)
    x = shared_batch(sizes, prefixes, [(37 * b) % 150 for b in range(B)], Hq=8, Hkv=2, d=d, ps=ps, dtype=DT[dtype], seed=8)
    dec = _decoder(x, dtype, ps)
    got = _call(dec, _cuda(x)).cpu().double()
    assert dec.last_error() == 0
    ref = dense64(x["q"], x["k_cache"], x["v_cache"], x["page_table"], x["seq_lens"])
    assert float(_row_errors(got, ref).max()) <= ROW_TOL
    dec.close()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B", [6, 50])
def test_shared_constant_values_come_back(dtype, d, B):
    # the weights' sum has to be that of the terms that meet the values: what each weight loses shows undiminished,
    # here with few keys that count (queries four times as long)
    x = shared_batch([B], [700], [(3 * b) % 60 for b in range(B)], Hq=8, Hkv=2, d=d, ps=16, dtype=DT[dtype], seed=9)
    x["q"] = x["q"] * 4
    value = 0.7109375
    x["v_cache"] = torch.where(x["v_cache"].isnan(), x["v_cache"], torch.full_like(x["v_cache"], value))
    dec = _decoder(x, dtype, 16)
    got = _call(dec, _cuda(x)).cpu().double()
    assert dec.last_error() == 0
    # 2^-16 of a weight, the truncation of six tiles' products and fp32 sums of 760 terms
    assert float((got / value - 1).abs().max()) <= 2**-15
    dec.close()


def _uniform_batch(B, heads, prefix, own, scale, *, d=64, ps=1024, seed=5):
    """bf16 sequences of equal length over one prefix in whole pages, on the GPU; keys of position p times scale(p)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    whole, more = prefix // ps, -(-own // ps)
    pages = whole + B * more
    k, v = (torch.empty(pages, heads, ps, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for c in (k, v):
        for p in range(0, pages, 64):
            c[p:p + 64] = torch.randn(c[p:p + 64].shape, generator=g, device="cuda").bfloat16()
    i32 = dict(dtype=torch.int32, device="cuda")
    table = torch.cat([torch.arange(whole, **i32).expand(B, whole),
                       whole + torch.arange(B * more, **i32).view(B, more)], 1).contiguous()
    for b in range(B) if own else range(1):
        first = 0 if b == 0 else whole
        for slot in range(first, whole + more):
            pos = slot * ps + torch.arange(ps, device="cuda")
            page = int(table[b, slot])
            k[page] = (k[page].float() * scale(pos.float())[:, None]).bfloat16()
    return dict(q=torch.randn(B, heads, d, generator=g, device="cuda").bfloat16(), k_cache=k, v_cache=v, page_table=table,
                seq_lens=torch.full((B,), prefix + own, **i32), group_start=torch.tensor([0, B], **i32),
                prefix_lens=torch.tensor([prefix], **i32), num_pages=pages, max_ctx=(whole + more) * ps)


@pytest.mark.gpu
@pytest.mark.parametrize("B,heads,prefix,own,period", [
    (3, 16, 102400, 5, 102400), (140, 16, 40960, 3, 40960), (2, 2, 130048, 1, 130048),  # long prefixes
    (64, 8, 0, 8000, 656),    # own parts of more chunks than one accumulator takes (64 * 500 * 8 over 6 * 1036 places)
    (32, 8, 4096, 16000, 700)])
def test_shared_long_parts_are_precise(B, heads, prefix, own, period):
    # scores that rise along every period, so that the maximum moves behind the first accumulators
    x = _uniform_batch(B, heads, prefix, own, lambda pos: 0.5 + 1.5 * (pos % period) / period)
    dec = _decoder(x, "bf16", 1024)
    got = _call(dec, x).double()
    assert dec.last_error() == 0
    ref = dense64(x["q"], x["k_cache"], x["v_cache"], x["page_table"], x["seq_lens"])
    assert float(_row_errors(got, ref).max()) <= ROW_TOL
    x["v_cache"].fill_(0.7109375)
    got = _call(dec, x).double() / 0.7109375
    assert float((got - 1).abs().max()) <= 2**-15
    dec.close()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_shared_captured_call_follows_new_groups(dtype):
    x = shared_batch([6, 5], [300, 130], [(5 * b) % 20 for b in range(11)], Hq=8, Hkv=2, d=64, ps=16, dtype=DT[dtype])
    dec = _decoder(x, dtype, 16)
    y = _cuda(x)
    out = torch.zeros(11, 8, 64, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _call(dec, y, out=out)
    ref = dense64(x["q"], x["k_cache"], x["v_cache"], x["page_table"], x["seq_lens"])
    # other groups over the same contents: shorter prefixes, one more sequence or fewer in the first group, no prefix
    for start, prefixes in (([0, 6, 11], [300, 130]), ([0, 6, 11], [77, 130]), ([0, 3, 11], [300, 0]),
                            ([0, 0, 11], [40, 0]), ([0, 5, 11], [299, 0])):
        y["group_start"].copy_(torch.tensor(start, dtype=torch.int32))
        y["prefix_lens"].copy_(torch.tensor(prefixes, dtype=torch.int32))
        out.fill_(float("nan"))
        graph.replay()
        assert float(_row_errors(out.cpu().double(), ref).max()) <= ROW_TOL, (start, prefixes)
        assert dec.last_error() == 0
    # lengths too: two sequences of the first group end before its prefix
    lens = x["seq_lens"].clone()
    lens[1], lens[4] = 20, 0
    y["seq_lens"].copy_(lens)
    y["group_start"].copy_(x["group_start"])
    y["prefix_lens"].copy_(x["prefix_lens"])
    graph.replay()
    ref = dense64(x["q"], x["k_cache"], x["v_cache"], x["page_table"], lens)
    assert float(_row_errors(out.cpu().double(), ref).max()) <= ROW_TOL and not out[4].any()
    assert dec.last_error() == 0
    dec.close()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_shared_sparse_and_dense_decodes_of_one_context(dtype):
    # they have the same workspace, one after the other, whatever each leaves there
    x = shared_batch([7, 5], [900, 400], [(41 * b) % 300 for b in range(12)], Hq=8, Hkv=2, d=64, ps=16, dtype=DT[dtype],
                     seed=12, garbage=0.0)
    y = _cuda(x)
    bad = dict(y, q=torch.full_like(y["q"], float("nan")))
    params = SparseDecoder.make_params(sinks=4, window=16, topk_abs=40, pilot_min=32, eps=0.05, delta=0.1, seed=3,
                                       num_pages=x["num_pages"])

    def caches(z):
        return z["q"], z["k_cache"], z["v_cache"], z["page_table"], z["seq_lens"]

    def sparse(dec, z):
        res = dec.decode(*caches(z), params)
        n = torch.arange(x["max_ctx"], device="cuda") < res["sel_count"][..., None]
        return [res["out"], torch.where(n, res["sel_idx"], -1), res["sel_count"], res["budgets"], res["head_need"]]

    calls = [sparse, lambda dec, z: [_call(dec, z)], lambda dec, z: [dec.dense(*caches(z), x["num_pages"])]]
    want = []
    for call in calls:
        dec = _decoder(x, dtype, 16)
        want.append(call(dec, y))
        dec.close()
    dec = _decoder(x, dtype, 16)
    for order in ([0, 1, 2], [2, 1, 0], [1, 0, 1, 2, 0, 2, 1]):
        for i in order:
            assert all(torch.equal(a, b) for a, b in zip(calls[i](dec, y), want[i])), (order, i)
        for i in order:                     # what follows is not to see what these leave
            calls[i](dec, bad)
    for i in (0, 1, 2, 1, 0):
        assert all(torch.equal(a, b) for a, b in zip(calls[i](dec, y), want[i])), i
    assert dec.last_error() == 0
    dec.close()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("batch,max_ctx", [(1, 32768), (64, 32768), (4096, 2048)])
def test_shared_records_take_no_more_than_the_sparse_decodes_scratch(dtype, batch, max_ctx):
    # keys and scores, 4 (1 + G) bytes per unit and position, and under 10 KB per unit and 16 MB of records and state
    # for the rest; the shared prefixes' records (about 17 to 166 MB) are within the former or nearly so
    Hq, Hkv = 32, 8
    dec = SparseDecoder(num_q_heads=Hq, num_kv_heads=Hkv, head_dim=128, dtype=DT[dtype], page_size=16, max_batch=batch,
                        max_ctx=max_ctx)
    units = batch * Hkv
    assert _abi.vattn_workspace_bytes(dec.ctx) <= units * max_ctx * 4 * (1 + Hq // Hkv) + units * 20480 + (16 << 20)
    dec.close()


@pytest.mark.gpu
def test_shared_accumulators_of_many_steps_lose_nothing_more():
    # 64 heads x 800 key tiles: about 170 steps of each stage. The tensor core loses up to 1.7e-8 with each of a
    # step's 16 products, 7e-6 between two records; weights of two terms and fp32 sums at random signs 1e-6 each. One
    # accumulator for all steps would be 3e-5 off.
    x = _uniform_batch(3, 64, 102400, 5, lambda pos: torch.ones_like(pos))
    x["v_cache"].fill_(0.7109375)
    dec = _decoder(x, "bf16", 1024)
    got = _call(dec, x).double() / 0.7109375
    assert dec.last_error() == 0
    assert float((got - 1).abs().max()) <= 2**-16
    dec.close()


@pytest.mark.gpu
@pytest.mark.parametrize("handle", [False, True])
def test_new_outputs_of_another_stream_leave_the_current_ones_memory(handle):
    # memory that the current stream has freed, and still reads, is not what a call on another stream writes to
    x = shared_batch([64], [600], [b for b in range(64)], Hq=32, Hkv=8, d=128, ps=16, dtype=torch.float32)
    dec = _decoder(x, "f32", 16)
    y = _cuda(x)
    r = Rotary(head_dim=128)
    other = torch.cuda.Stream()
    stream = other.cuda_stream if handle else other
    one = torch.arange(64, dtype=torch.int32, device="cuda")
    k, v = (torch.randn(64, 8, 128, device="cuda") for _ in range(2))
    spare = {n: torch.zeros_like(y[n]) for n in ("k_cache", "v_cache")}
    calls = [lambda **kw: r.rotate(y["q"], one, **kw), lambda **kw: _call(dec, y, **kw),
             lambda **kw: dec.append(k, v, spare["k_cache"], spare["v_cache"], y["page_table"], y["seq_lens"],
                                     x["num_pages"], rotary=r, q=y["q"], **kw)]
    for call in calls:
        want = call().clone()
        torch.cuda.synchronize()
        held = torch.full_like(want, 3.0)
        torch.cuda.synchronize()
        torch.cuda._sleep(20_000_000)           # 10 ms of the current stream
        seen = held * 2
        del held
        got = call(stream=stream)
        torch.cuda.synchronize()
        assert (seen == 6).all() and torch.equal(got, want)
        del got, seen
    dec.close()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("groups", [20, 1100])
def test_shared_many_groups_behind_short_first_sequences(dtype, groups):
    # in every group one of two sequences reaches the prefix's end, mostly the second, which does not list its pages
    prefixes = [20 + g % 40 for g in range(groups)]
    own = [v for g in range(groups) for v in ((-3, g % 7) if g % 3 else (g % 5, -4))]
    x = shared_batch([2] * groups, prefixes, own, Hq=4, Hkv=2, d=64, ps=16, dtype=DT[dtype], seed=15)
    ref = dense64(x["q"], x["k_cache"], x["v_cache"], x["page_table"], x["seq_lens"])
    table = x["page_table"].clone()
    for g in range(groups):
        if g % 3:
            table[2 * g + 1, :prefixes[g] // 16] = -1
    dec = _decoder(x, dtype, 16)
    got = _call(dec, _cuda(dict(x, page_table=table))).cpu().double()
    assert dec.last_error() == 0
    assert float(_row_errors(got, ref).max()) <= ROW_TOL
    dec.close()


# ------------------------------------------------------------ as they are used together
@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_serving_steps(dtype):
    """Append a shared prompt once, then decode steps: append with rotation, shared decode, sparse decode."""
    dt, d, Hq, Hkv, ps, B, prompt, steps = DT[dtype], 64, 8, 2, 16, 5, 75, 4
    g = torch.Generator().manual_seed(11)
    rotary = Rotary(head_dim=d, rot_dim=32, scaling="linear", factor=2.0)
    freq = frequencies(32, scaling="linear", factor=2.0)
    max_ctx = prompt + steps
    pps = -(-max_ctx // ps)
    whole = prompt // ps
    # every sequence lists the prompt's whole pages, and pages of its own behind them
    table = torch.zeros(B, pps, dtype=torch.int32)
    table[:, :whole] = torch.arange(whole)
    table[:, whole:] = whole + torch.arange(B * (pps - whole)).view(B, -1)
    pages = whole + B * (pps - whole)
    i32 = dict(dtype=torch.int32, device="cuda")
    k_cache = torch.full((pages, Hkv, ps, d), float("nan"), dtype=dt, device="cuda")
    v_cache = torch.full((pages, Hkv, ps, d), float("nan"), dtype=dt, device="cuda")
    dec = SparseDecoder(num_q_heads=Hq, num_kv_heads=Hkv, head_dim=d, dtype=dt, page_size=ps, max_batch=B,
                        max_ctx=max_ctx)
    K = torch.randn(prompt, Hkv, d, generator=g).to(dt)
    V = torch.randn(prompt, Hkv, d, generator=g).to(dt)
    tab = table.cuda()
    # the prompt once into sequence 0's pages; the page it ends in copied to the others'
    dec.append(K.cuda(), V.cuda(), k_cache, v_cache, tab[:1], torch.tensor([prompt], **i32), pages,
               cu_tokens=torch.tensor([0, prompt], **i32), rotary=rotary)
    for c in (k_cache, v_cache):
        c[tab[1:, whole].long()] = c[tab[0, whole].long()].clone()
    hist_k = [rotate64(K, torch.arange(prompt), 32, "half", freq).to(dt)] * B
    hist_v = [V] * B
    seq_lens = torch.full((B,), prompt, **i32)
    group_start, prefix = torch.tensor([0, B], **i32), torch.tensor([prompt], **i32)
    for step in range(steps):
        seq_lens += 1
        q, k, v = (torch.randn(B, h, d, generator=g).to(dt) for h in (Hq, Hkv, Hkv))
        qr = dec.append(k.cuda(), v.cuda(), k_cache, v_cache, tab, seq_lens, pages, rotary=rotary, q=q.cuda())
        shared = dec.shared_dense(qr, k_cache, v_cache, tab, seq_lens, pages, group_start, prefix)
        params = SparseDecoder.make_params(sinks=4, window=max_ctx, eps=0.1, delta=0.1, seed=0, num_pages=pages)
        sparse = dec.decode(qr, k_cache, v_cache, tab, seq_lens, params)["out"]   # the window covers everything
        assert dec.last_error() == 0
        pos = torch.full((B,), prompt + step)
        kr, q64 = rotate64(k, pos, 32, "half", freq), rotate64(q, pos, 32, "half", freq)
        hist_k = [torch.cat([h, kr[b:b + 1].to(dt)]) for b, h in enumerate(hist_k)]
        hist_v = [torch.cat([h, v[b:b + 1]]) for b, h in enumerate(hist_v)]
        for b in range(B):
            s = q64[b].to(dt).double().view(Hkv, -1, d) @ hist_k[b].double().permute(1, 2, 0) / math.sqrt(d)
            ref = (torch.softmax(s, -1) @ hist_v[b].double().transpose(0, 1)).reshape(Hq, d)
            # the rotated rows may round to the neighbouring value where fp32 and 64 bits straddle a tie:
            # half an ulp (bf16 2^-9 of a product at most, 16 of them at random signs) of a score
            tol = (2**-6 if dtype == "bf16" else 2**-14) * float(V.float().abs().max())
            assert float((shared[b].cpu().double() - ref).abs().max()) <= tol
            assert float((sparse[b].cpu().double() - ref).abs().max()) <= tol
    dec.close()
