"""Convenience wrapper over the C ABI: one context plus its output buffers.

Marshalling only — every step runs in libvattn.so. Tensors are torch CUDA
tensors in the layouts of include/vattn.h.
"""
import torch

from . import _abi

_DTYPES = {torch.float32: _abi.VATTN_FP32, torch.bfloat16: _abi.VATTN_BF16}
_PROXIES = {"exact": _abi.VATTN_EXACT, "sparq": _abi.VATTN_SPARQ, "loki": _abi.VATTN_LOKI}
_GUARANTEES = {"denominator": _abi.VATTN_GUARANTEE_DENOMINATOR, "output": _abi.VATTN_GUARANTEE_OUTPUT}
# "host": k_cache and v_cache are page-locked host tensors (tensor.pin_memory())
_KV = {"device": _abi.VATTN_KV_DEVICE, "host": _abi.VATTN_KV_HOST}


class SparseDecoder:
    """A vattn context for fixed shapes (see vattn_config in include/vattn.h)."""

    def __init__(self, *, num_q_heads, num_kv_heads, head_dim, dtype, page_size, max_batch,
                 max_ctx, proxy="exact", proxy_rank=0, device=None, kv_location="device"):
        self.device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
        self.num_q_heads, self.num_kv_heads, self.head_dim = num_q_heads, num_kv_heads, head_dim
        self.max_batch, self.max_ctx, self.page_size = max_batch, max_ctx, page_size
        self.pages_per_seq = -(-max_ctx // page_size)
        # the device index of the caches (-1: page-locked host memory) and of everything else
        self._index = torch.cuda.current_device() if self.device.index is None else self.device.index
        self._cache_index = -1 if kv_location == "host" else self._index
        self._cache_shape = (num_kv_heads, page_size, head_dim)
        self.proxy = proxy
        self.dtype = dtype
        cfg = _abi.vattn_config(num_q_heads=num_q_heads, num_kv_heads=num_kv_heads,
                                head_dim=head_dim, dtype=_DTYPES[dtype], page_size=page_size,
                                max_batch=max_batch, max_ctx=max_ctx, proxy=_PROXIES[proxy],
                                proxy_rank=proxy_rank, kv_location=_KV[kv_location])
        with torch.cuda.device(self.device):
            self.ctx = _abi.vattn_create(cfg)

    def alloc_outputs(self, batch):
        dev = self.device
        return dict(
            out=torch.empty((batch, self.num_q_heads, self.head_dim), dtype=torch.float32, device=dev),
            sel_idx=torch.empty((batch, self.num_kv_heads, self.max_ctx), dtype=torch.int32, device=dev),
            sel_count=torch.empty((batch, self.num_kv_heads), dtype=torch.int32, device=dev),
            budgets=torch.empty((batch, self.num_kv_heads), dtype=torch.int32, device=dev),
            head_need=torch.empty((batch, self.num_q_heads), dtype=torch.int32, device=dev))

    @staticmethod
    def make_params(*, sinks, window, topk_abs=0, topk_num=0, topk_den=0, pilot_min=64,
                    pilot_num=0, pilot_den=0, eps, delta, seed, num_pages, k_t_cache=None,
                    k_proj_cache=None, proj_basis=None, guarantee="denominator", topp_num=0,
                    topp_den=0, batch_offset=0, head_offset=0):
        return _abi.vattn_params(
            sinks=sinks, window=window, topk_abs=topk_abs, topk_num=topk_num, topk_den=topk_den,
            pilot_min=pilot_min, pilot_num=pilot_num, pilot_den=pilot_den, eps=eps, delta=delta,
            seed=seed, num_pages=num_pages,
            k_t_cache=None if k_t_cache is None else k_t_cache.data_ptr(),
            k_proj_cache=None if k_proj_cache is None else k_proj_cache.data_ptr(),
            proj_basis=None if proj_basis is None else proj_basis.data_ptr(),
            guarantee=_GUARANTEES[guarantee], topp_num=topp_num, topp_den=topp_den,
            batch_offset=batch_offset, head_offset=head_offset)

    def decode(self, q, k_cache, v_cache, page_table, seq_lens, params, outputs=None, stream=None):
        batch = q.shape[0]
        o = outputs if outputs is not None else self.alloc_outputs(batch)
        _abi.vattn_decode(self.ctx, q, k_cache, v_cache, page_table, seq_lens, batch, params,
                          o["out"], o["sel_idx"], o["sel_count"], o["budgets"], o["head_need"],
                          stream=stream)
        return o

    def dense(self, q, k_cache, v_cache, page_table, seq_lens, num_pages, out=None, stream=None):
        batch = q.shape[0]
        if out is None:
            out = torch.empty((batch, self.num_q_heads, self.head_dim), dtype=torch.float32,
                              device=self.device)
        _abi.vattn_dense_decode(self.ctx, q, k_cache, v_cache, page_table, seq_lens, batch,
                                num_pages, out, stream=stream)
        return out

    def _stream(self, stream):
        # the context's device's current stream (the raw handle: no stream object is made per call)
        return torch._C._cuda_getCurrentRawStream(self._index) if stream is None else stream

    def _check_cache(self, name, t, num_pages, shape, index):
        if t is None or t.dtype is not self.dtype or t.shape[1:] != shape or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous {self.dtype} [pages, {', '.join(map(str, shape))}] tensor")
        if t.shape[0] < num_pages:
            raise ValueError(f"{name} holds {t.shape[0]} pages, num_pages is {num_pages}")
        if t.get_device() != index:
            raise ValueError(f"{name} is on {t.device}, the context's caches on "
                             f"{self.device if index >= 0 else 'the host'}")

    def _check_index(self, name, t, shape):
        if t.dtype is not torch.int32 or t.shape != shape or not t.is_contiguous() or t.get_device() != self._index:
            raise ValueError(f"{name} must be a contiguous int32 {list(shape)} tensor on {self.device}")

    def _check_caches(self, k_cache, v_cache, page_table, seq_lens, num_pages):
        """The caches, table and lengths of one call; returns its batch."""
        batch = seq_lens.shape[0]
        shape = self._cache_shape
        self._check_cache("k_cache", k_cache, num_pages, shape, self._cache_index)
        self._check_cache("v_cache", v_cache, num_pages, shape, self._cache_index)
        if batch > self.max_batch:
            raise ValueError(f"a batch of {batch} in a context for {self.max_batch}")
        self._check_index("page_table", page_table, (batch, self.pages_per_seq))
        self._check_index("seq_lens", seq_lens, (batch,))
        return batch

    def _check_rows(self, name, t, tokens, heads):
        if t.dtype is not self.dtype or t.shape != (tokens, heads, self.head_dim) or t.stride(2) != 1 \
                or (heads > 1 and t.stride(1) != self.head_dim) or t.get_device() != self._index:
            raise ValueError(f"{name} must be {self.dtype} [{tokens}, {heads}, {self.head_dim}] on {self.device} with "
                             "the heads of a token contiguous")
        # a single token's stride says nothing: its row is contiguous, a view of a wider one too
        return heads * self.head_dim if tokens <= 1 else t.stride(0)

    def append(self, k, v, k_cache, v_cache, page_table, seq_lens, num_pages, *, cu_tokens=None, rotary=None, q=None,
               q_out=None, k_t_cache=None, k_proj_cache=None, proj_basis=None, stream=None):
        """Write new tokens' keys (rotated) and values into the caches; rotate their queries.

        k, v [tokens, Hkv, d] and q [tokens, Hq, d] may be views with a larger token
        stride (a fused projection). seq_lens counts the new tokens already. cu_tokens
        [batch + 1]: the tokens of sequence b are cu_tokens[b] .. cu_tokens[b+1]-1; None:
        one token per sequence (none where the length is 0). A SparQ context also takes
        k_t_cache, a Loki context k_proj_cache and proj_basis. Returns q_out, new and
        contiguous by default (None without q). Autograd records nothing of the call;
        see vattn_append in include/vattn.h.
        """
        batch = self._check_caches(k_cache, v_cache, page_table, seq_lens, num_pages)
        tokens = k.shape[0]
        p = _abi.vattn_append_params()
        p.tokens, p.num_pages = tokens, num_pages
        p.k_stride = self._check_rows("k", k, tokens, self.num_kv_heads)
        p.v_stride = self._check_rows("v", v, tokens, self.num_kv_heads)
        p.k, p.v, p.k_cache, p.v_cache = k.data_ptr(), v.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr()
        if q is not None:
            p.q_stride = self._check_rows("q", q, tokens, self.num_q_heads)
            if q_out is None:
                q_out = _abi.empty_for(stream, (tokens, self.num_q_heads, self.head_dim), dtype=self.dtype,
                                       device=self.device)
            elif self._check_rows("q_out", q_out, tokens, self.num_q_heads) != self.num_q_heads * self.head_dim:
                raise ValueError("q_out must be contiguous")
            p.q, p.q_out = q.data_ptr(), q_out.data_ptr()
        else:
            q_out = None
        if cu_tokens is not None:
            self._check_index("cu_tokens", cu_tokens, (batch + 1,))
            p.cu_tokens = cu_tokens.data_ptr()
        elif tokens != batch:
            raise ValueError(f"{tokens} tokens for {batch} sequences need cu_tokens")
        if rotary is not None:
            if rotary.head_dim != self.head_dim:
                raise ValueError(f"a rotation of {rotary.head_dim} components for heads of {self.head_dim}")
            p.rope = _abi.C.pointer(rotary.plan)
        if self.proxy == "sparq":
            self._check_cache("k_t_cache", k_t_cache, num_pages, (self.num_kv_heads, self.head_dim, self.page_size),
                              self._index)
            p.k_t_cache = k_t_cache.data_ptr()
        elif self.proxy == "loki":
            self._check_cache("k_proj_cache", k_proj_cache, num_pages, (self.num_kv_heads, self.page_size, 32),
                              self._index)
            if proj_basis is None or proj_basis.dtype is not torch.float32 or not proj_basis.is_contiguous() \
                    or proj_basis.shape != (self.num_kv_heads, self.head_dim, 32) \
                    or proj_basis.get_device() != self._index:
                raise ValueError(f"proj_basis must be contiguous float32 [{self.num_kv_heads}, {self.head_dim}, 32] "
                                 f"on {self.device}")
            p.k_proj_cache, p.proj_basis = k_proj_cache.data_ptr(), proj_basis.data_ptr()
        _abi.vattn_append(self.ctx, p, page_table, seq_lens, batch, self._stream(stream))
        return q_out

    def shared_dense(self, q, k_cache, v_cache, page_table, seq_lens, num_pages, group_start, prefix_lens, out=None,
                     stream=None):
        """dense() for a batch whose groups of sequences share prefixes, each read once.

        group_start [groups + 1], prefix_lens [groups] int32: the first prefix_lens[g]
        positions of sequences group_start[g] .. group_start[g+1]-1 hold the same keys
        and values, read through the pages of the group's first sequence; see
        vattn_shared_dense_decode in include/vattn.h.
        """
        batch = self._check_caches(k_cache, v_cache, page_table, seq_lens, num_pages)
        if q.dtype is not self.dtype or q.shape != (batch, self.num_q_heads, self.head_dim) \
                or not q.is_contiguous() or q.get_device() != self._index:
            raise ValueError(f"q must be contiguous {self.dtype} [{batch}, {self.num_q_heads}, {self.head_dim}] "
                             f"on {self.device}")
        groups = prefix_lens.shape[0]
        self._check_index("prefix_lens", prefix_lens, (groups,))
        self._check_index("group_start", group_start, (groups + 1,))
        if out is None:
            out = _abi.empty_for(stream, (batch, self.num_q_heads, self.head_dim), dtype=torch.float32,
                                 device=self.device)
        elif out.dtype is not torch.float32 or out.shape != q.shape or not out.is_contiguous() \
                or out.get_device() != self._index:
            raise ValueError(f"out must be contiguous float32 {list(q.shape)} on {self.device}")
        _abi.vattn_shared_dense_decode(self.ctx, q, k_cache, v_cache, page_table, seq_lens, group_start, prefix_lens,
                                       groups, batch, num_pages, out, stream=self._stream(stream))
        return out

    def last_error(self, sync=True):
        return _abi.vattn_last_error(self.ctx, sync)

    def close(self):
        if getattr(self, "ctx", None):
            _abi.vattn_destroy(self.ctx)
            self.ctx = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def decoder_for(w, device=None, max_batch=None, kv_location="device"):
    """A SparseDecoder shaped for a synthetic workload description (synth.Workload)."""
    dt = torch.float32 if w.dtype == "f32" else torch.bfloat16
    return SparseDecoder(num_q_heads=w.num_q_heads, num_kv_heads=w.num_kv_heads,
                         head_dim=w.head_dim, dtype=dt, page_size=w.page_size,
                         max_batch=w.batch if max_batch is None else max_batch, max_ctx=w.max_ctx,
                         proxy=w.proxy, proxy_rank=w.proxy_rank, device=device,
                         kv_location=kv_location)


def params_for(w, inputs, eps=None, seed=None, guarantee=None, batch_offset=0, head_offset=0):
    """vattn_params of a synthetic workload with its drawn inputs (device tensors); the
    offsets place a shard of a larger batch."""
    return SparseDecoder.make_params(
        sinks=w.sinks, window=w.window, topk_abs=w.topk_abs, topk_num=w.topk_num,
        topk_den=w.topk_den, pilot_min=w.pilot_min, pilot_num=w.pilot_num, pilot_den=w.pilot_den,
        eps=w.eps if eps is None else eps, delta=w.delta, seed=w.seed if seed is None else seed,
        num_pages=int(inputs["num_pages"]), k_t_cache=inputs.get("k_t_cache"),
        k_proj_cache=inputs.get("k_proj_cache"), proj_basis=inputs.get("proj_basis"),
        guarantee=guarantee or w.guarantee, topp_num=w.topp_num, topp_den=w.topp_den,
        batch_offset=batch_offset, head_offset=head_offset)
