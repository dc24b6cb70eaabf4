"""Torch-facing 4-bit KV cache (argument checks and marshalling).

PyTorch holds the buffers and gives the current stream; the work is done by the
library's kernels through the C ABI (include/sa.h: sa_kv4_*).
"""

import torch

from . import _binding as B

_DTYPES = {torch.bfloat16: B.SA_DTYPE_BF16, torch.float16: B.SA_DTYPE_FP16}


class QuantKVCache:
    """Keys and values of ``batch`` sequences, 4.5 bits a value, with the attention weight
    each row has drawn.

    Tensors are bf16 or fp16 [B, T, heads, D] on the cache's device, D contiguous, the other
    strides multiples of 8 (a slice of a fused projection will do). K and Q come with
    their position encoding applied. ``counts`` (int32 [B] on the device, or None for T each)
    gives the valid tokens of each sequence of a padded batch. For serving: no call records
    gradients.

    The buffers are attributes: ``k_codes``, ``v_codes`` [B, Hk, N, D / 2] and
    ``k_scales``, ``v_scales`` [B, Hk, N, D / 16] (uint8), ``pos`` (int32) and ``weight``
    (fp32) [B, Hk, N], ``seq`` (int32 [4, B]: rows held, rows appended in all, rows of the
    last append, rows appended since the last eviction) and ``status`` (int32 [4]).

    One workspace serves every call; calls on one cache, replays of captured ones among
    them, must be ordered (one stream, or events). Before capturing a graph make one call
    of the same shape, so that the workspace is there; the object must live as long as
    the graphs captured from its calls.
    """

    def __init__(self, batch, kv_heads, head_dim, capacity, device=None):
        dev = torch.device("cuda", torch.cuda.current_device()) if device is None \
            else torch.device(device)
        if capacity < 1 or capacity % 128:
            raise ValueError("capacity must be a positive multiple of 128")
        planes = (batch, kv_heads, capacity)
        u8 = dict(dtype=torch.uint8, device=dev)
        self._set(k_codes=torch.empty(planes + (head_dim // 2,), **u8),
                  v_codes=torch.empty(planes + (head_dim // 2,), **u8),
                  k_scales=torch.empty(planes + (head_dim // 16,), **u8),
                  v_scales=torch.empty(planes + (head_dim // 16,), **u8),
                  pos=torch.empty(planes, dtype=torch.int32, device=dev),
                  weight=torch.empty(planes, dtype=torch.float32, device=dev),
                  seq=torch.zeros((4, batch), dtype=torch.int32, device=dev),
                  status=torch.zeros(4, dtype=torch.int32, device=dev))

    @classmethod
    def from_tensors(cls, k_codes, v_codes, k_scales, v_scales, pos, weight, seq, status):
        """A cache over buffers that exist already (of the shapes above)."""
        self = cls.__new__(cls)
        self._set(k_codes=k_codes, v_codes=v_codes, k_scales=k_scales, v_scales=v_scales,
                  pos=pos, weight=weight, seq=seq, status=status)
        return self

    def _set(self, **tensors):
        codes = tensors["k_codes"]
        if codes.dim() != 4:
            raise ValueError("k_codes must be [batch, kv_heads, capacity, head_dim / 2]")
        b, h, n, half = codes.shape
        self.batch, self.kv_heads, self.capacity, self.head_dim = b, h, n, 2 * half
        self.device = codes.device
        if self.device.type != "cuda":
            raise ValueError(f"the cache must be on a GPU, not on {self.device}")
        self._index = codes.device.index
        want = {"k_codes": (torch.uint8, (b, h, n, half)),
                "v_codes": (torch.uint8, (b, h, n, half)),
                "k_scales": (torch.uint8, (b, h, n, half // 8)),
                "v_scales": (torch.uint8, (b, h, n, half // 8)),
                "pos": (torch.int32, (b, h, n)), "weight": (torch.float32, (b, h, n)),
                "seq": (torch.int32, (4, b)), "status": (torch.int32, (4,))}
        for name, (dtype, shape) in want.items():
            t = tensors[name]
            if t.dtype != dtype or tuple(t.shape) != shape or not t.is_contiguous() \
                    or t.device != self.device:
                raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {shape} "
                                 f"on {self.device}")
            setattr(self, name, t)
        self._c = B.SaKv4Cache(b, h, self.head_dim, n,
                               *(tensors[f].data_ptr() for f, _ in B.SaKv4Cache._fields_[4:]))
        self._workspaces = []
        self._sizes = {}

    # -- helpers
    def _rows(self, t, name, tokens, heads, dtype):
        if t.shape != (self.batch, tokens, heads, self.head_dim) or t.dtype != dtype \
                or t.device != self.device or t.stride(3) != 1:
            raise ValueError(f"{name} must be a {dtype} tensor of shape "
                             f"{(self.batch, tokens, heads, self.head_dim)} on {self.device} "
                             f"with contiguous rows")
        sb, st, sh, _ = t.stride()
        # torch leaves the stride of a dimension of size 1 open
        return B.SaRows(t.data_ptr(), sb if self.batch > 1 else 0, st if tokens > 1 else 0,
                        sh if heads > 1 else 0)

    def _tokens_heads(self, t, name):
        if t.dim() != 4 or t.dtype not in _DTYPES:
            raise ValueError(f"{name} must be a bf16 or fp16 tensor [batch, tokens, heads, "
                             f"head_dim]")
        return t.shape[1], t.shape[2]

    def _counts(self, counts):
        if counts is None:
            return 0
        if counts.dtype != torch.int32 or counts.shape != (self.batch,) \
                or counts.device != self.device or not counts.is_contiguous():
            raise ValueError(f"counts must be a contiguous int32 tensor of shape "
                             f"{(self.batch,)} on {self.device}")
        return counts.data_ptr()

    def _stream(self, stream):
        # the raw handle: making a Stream object costs more than the rest of a call's checks
        return torch._C._cuda_getCurrentRawStream(self._index) if stream is None \
            else stream.cuda_stream

    def _empty(self, shape, dtype, stream):
        # memory of the stream that writes it: another's may still be in use there
        with torch.cuda.device(self.device), torch.cuda.stream(stream):
            return torch.empty(shape, dtype=dtype, device=self.device)

    def _work(self, key, nbytes, stream):
        """(pointer, bytes) of a workspace of at least `nbytes()`. One that became too small
        stays allocated: a captured graph, or a call under way on another stream, may use it.
        Each is at least twice the one before, so all together are less than twice the last.
        (0, 0) for a call that needs none, or is refused for its sizes (the library says why)."""
        need = self._sizes.get(key)
        if need is None:
            need = self._sizes[key] = nbytes()
        if need == 0:
            return 0, 0
        have = self._workspaces[-1].numel() if self._workspaces else 0
        if have < need:
            with torch.cuda.device(self.device), torch.cuda.stream(stream):
                capturing = torch.cuda.is_current_stream_capturing()
            if capturing:
                raise RuntimeError("make one call of this shape before capturing it: the "
                                   "workspace is too small")
            self._workspaces.append(self._empty(max(need, 2 * have), torch.uint8, stream))
        last = self._workspaces[-1]
        return last.data_ptr(), last.numel()

    # -- the calls
    def append(self, K, V, counts=None, replace=False, stream=None):
        """Quantise rows of K and V [B, T, Hk, D] behind the rows held; with ``replace`` in
        place of the rows of the last append."""
        tokens, _ = self._tokens_heads(K, "K")
        k = self._rows(K, "K", tokens, self.kv_heads, K.dtype)
        v = self._rows(V, "V", tokens, self.kv_heads, K.dtype)
        B.sa_kv4_append(self._c, k, v, _DTYPES[K.dtype], tokens, self._counts(counts), replace,
                        self._stream(stream))

    def read(self, first, K, V, stream=None):
        """Stored values of rows first .. first + T - 1 into K, V [B, T, Hk, D]; rows not held
        leave them as they are."""
        tokens, _ = self._tokens_heads(K, "K")
        k = self._rows(K, "K", tokens, self.kv_heads, K.dtype)
        v = self._rows(V, "V", tokens, self.kv_heads, K.dtype)
        B.sa_kv4_read(self._c, first, k, v, _DTYPES[K.dtype], tokens, self._stream(stream))

    def read_last(self, K, V, stream=None):
        """Stored values of the rows of the last append into K, V [B, T, Hk, D]."""
        self.read(B.SA_KV4_LAST, K, V, stream)

    def attend(self, Q, counts=None, causal=False, scale=0.0, out=None, lse=None,
               add_weight=False, stream=None):
        """Attention of Q [B, T, heads, D] over the rows held (``causal``: the queries are
        those of the last rows appended); returns ``out``. ``lse``: fp32 [B, heads, T] or None.
        ``add_weight`` adds the probabilities each row drew to ``weight``."""
        tokens, heads = self._tokens_heads(Q, "Q")
        if heads < 1 or heads % self.kv_heads:
            raise ValueError(f"Q must have a multiple of {self.kv_heads} heads")
        if out is None:
            out = self._empty(Q.shape, Q.dtype, stream) if stream is not None \
                else torch.empty(Q.shape, dtype=Q.dtype, device=self.device)
        q = self._rows(Q, "Q", tokens, heads, Q.dtype)
        o = self._rows(out, "out", tokens, heads, Q.dtype)
        lse_ptr = 0
        if lse is not None:
            if lse.dtype != torch.float32 or lse.shape != (self.batch, heads, tokens) \
                    or not lse.is_contiguous() or lse.device != self.device:
                raise ValueError(f"lse must be contiguous fp32 of shape "
                                 f"{(self.batch, heads, tokens)} on {self.device}")
            lse_ptr = lse.data_ptr()
        ws, nbytes = self._work(("attend", heads, tokens, bool(add_weight)),
                                lambda: B.sa_kv4_attend_bytes(self._c, heads, tokens, add_weight),
                                stream)
        B.sa_kv4_attend(self._c, q, o, _DTYPES[Q.dtype], heads, tokens, self._counts(counts),
                        causal, scale, lse_ptr, add_weight, ws, nbytes, self._stream(stream))
        return out

    def evict(self, keep, first=0, recent=0, stream=None):
        """Evict every sequence down to ``keep`` rows per KV head: the first ``first`` and the
        last ``recent`` rows appended stay, of the others those of the largest weight."""
        ws, nbytes = self._work("evict", lambda: B.sa_kv4_evict_bytes(self._c), stream)
        B.sa_kv4_evict(self._c, keep, first, recent, ws, nbytes, self._stream(stream))

    def rows_held(self):
        """Rows each sequence holds (int32 [B], a view on the device)."""
        return self.seq[0]

    def reset(self, stream=None):
        """Forget every row and clear the status word."""
        B.sa_kv4_reset(self._c, self._stream(stream))

    def check(self, stream=None):
        """The status word as an sa_status (waits for the stream)."""
        return B.sa_kv4_get_status(self._c, self._stream(stream))
