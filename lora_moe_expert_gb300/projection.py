"""One MoE projection from hidden states to hidden states, the operators in their order.

``MoeProjection`` holds what a serving process keeps (the experts' weights, stacked; their 4-bit
form; the LoRA tables) and runs a batch through

* prefill: the router's top_k -> rows into expert order -> the expert GEMM with the LoRA fold in
  its epilogue -> rows back to their tokens, weighted;
* decode: the router's top_k -> the 4-bit product of every (token, slot) row -> the decode fold
  -> the weighted sum over a token's slots (the rows are in flat order, nothing is sorted);
* the gradient of prefill's dispatch, combine and router weights, for training a router over frozen
  experts: given the gradient of the output, those of the experts' rows and of the logits (the
  experts' own products and the fold have no gradient here).

torch provides device memory and streams only.

    python -m lora_moe_expert_gb300.projection     # runs both forms on random data
"""
from __future__ import annotations

import numpy as np
import torch

import lora_moe_expert_gb300 as mlg


def _i32(*shape):
    return torch.empty(*shape, dtype=torch.int32, device="cuda")


def _expect(what, t, shape, dtype=None):
    """A kernel reads `shape` from t's address, whatever t is."""
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{what}: {tuple(shape)} expected, {tuple(t.shape)} given")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{what}: {dtype} expected, {t.dtype} given")
    if not t.is_cuda:
        raise ValueError(f"{what}: on the GPU expected")


class MoeProjection:
    """n_experts experts, W_e [n_out, k_in]; lora: (ids, A, B, scale) with A [n, max_rank, k_in] and
    B [n, n_out, max_rank] bf16 of the adapted experts, or None; q4: (codes, scales, zeros, group)
    of the same weights, or None when decode is not wanted."""

    def __init__(self, weights, top_k: int, lora=None, q4=None, renormalize: bool = True):
        self.w = weights.contiguous()
        self.n_experts, self.n_out, self.k_in = self.w.shape
        E, bf16 = self.n_experts, torch.bfloat16
        _expect("weights", self.w, (E, self.n_out, self.k_in), bf16)
        self.top_k, self.renormalize, self.saved = top_k, renormalize, None
        self.q4 = None if q4 is None else self._four_bit(*q4)
        self.max_rank = 8 if lora is None else lora[1].shape[1]
        a, b, s = np.zeros(E, np.uint64), np.zeros(E, np.uint64), np.zeros(E, np.float32)
        if lora is not None:
            ids, self.A, self.B, scale = lora[0], lora[1].contiguous(), lora[2].contiguous(), lora[3]
            _expect("A", self.A, (len(ids), self.max_rank, self.k_in), bf16)
            _expect("B", self.B, (len(ids), self.n_out, self.max_rank), bf16)
            step_a, step_b = self.A[0].numel() * 2, self.B[0].numel() * 2
            pa, pb, ps = mlg.mlg_pack_expert_tables(
                ids, [self.A.data_ptr() + i * step_a for i in range(len(ids))],
                [self.B.data_ptr() + i * step_b for i in range(len(ids))], scale)
            a[:pa.size], b[:pb.size], s[:ps.size] = pa, pb, ps
        self.a_table = torch.empty(E, dtype=torch.int64, device="cuda")
        self.b_table = torch.empty(E, dtype=torch.int64, device="cuda")
        self.scale_table = torch.empty(E, dtype=torch.float32, device="cuda")
        mlg.mlg_upload_expert_tables(a, b, s, self.a_table, self.b_table, self.scale_table)

    def _four_bit(self, codes, scales, zeros, group):
        groups = (self.n_experts, self.n_out, self.k_in // group)
        _expect("codes", codes, (self.n_experts, self.n_out, self.k_in // 2), torch.uint8)
        _expect("scales", scales, groups, torch.bfloat16)
        if zeros is not None:
            _expect("zeros", zeros, groups, torch.uint8)
            if zeros.numel() > 0 and int(zeros.max()) > 15:
                raise ValueError("zeros: 0 to 15 expected (a format may store them less one)")
            zeros = zeros.contiguous()
        return codes.contiguous(), scales.contiguous(), zeros, group

    def _batch(self, x, logits, row_map):
        T = x.shape[0]
        _expect("x", x, (T, self.k_in), torch.bfloat16)
        _expect("logits", logits, (T, self.n_experts))
        if row_map is not None:
            _expect("row_map", row_map, (T,), torch.int32)
            row_map = row_map.contiguous()
        return row_map

    def route(self, logits):
        """(indices [tokens, top_k] int32, weights [tokens, top_k] float)."""
        T = logits.shape[0]
        indices = _i32(T, self.top_k)
        weights = torch.empty(T, self.top_k, device="cuda")
        mlg.mlg_route_topk(logits, indices, weights, T, self.n_experts, self.top_k,
                           self.renormalize)
        return indices, weights

    def prefill(self, x, logits, row_map=None, keep: bool = True):
        """x [tokens, k_in] bf16, logits [tokens, n_experts] -> [tokens, n_out] bf16; row_map
        [tokens] int32, negative for a token whose request uses no adapter (None: all use it).
        With keep, self.saved holds what backward() needs, the experts' rows among it (top_k times
        the output), until the next prefill(): one batch at a time.  Without, nothing is held."""
        row_map = self._batch(x, logits, row_map)
        T, K, n = x.shape[0], self.top_k, x.shape[0] * self.top_k
        indices, weights = self.route(logits)
        offsets, src, pos = _i32(self.n_experts + 1), _i32(n), _i32(n)
        x_rows = torch.empty(n, self.k_in, dtype=torch.bfloat16, device="cuda")
        y_rows = torch.empty(n, self.n_out, dtype=torch.bfloat16, device="cuda")
        out = torch.empty(T, self.n_out, dtype=torch.bfloat16, device="cuda")
        mlg.mlg_dispatch(x, indices, None, offsets, src, pos, x_rows, n, self.k_in, K,
                         self.n_experts)
        if n > 0:  # an empty batch has no rows' addresses to give
            mlg.mlg_grouped_gemm_fold_xrows(x_rows, offsets, src, row_map, self.w, self.a_table,
                                            self.b_table, self.scale_table, y_rows, self.k_in,
                                            self.max_rank, self.n_out, K, self.n_experts, 0, n, n)
        mlg.mlg_combine(y_rows, pos, weights, out, T, self.n_out, K, n)
        self.saved = (logits, indices, weights, offsets, pos, y_rows) if keep else None
        return out

    def _last(self):
        if self.saved is None:
            raise RuntimeError("no prefill() with keep before")
        return self.saved

    def backward(self, dout):
        """Gradients of the last prefill() with respect to the experts' rows (sorted order) and
        the logits, given that of its output."""
        logits, indices, weights, offsets, pos, y_rows = self._last()
        T, K, n = logits.shape[0], self.top_k, y_rows.shape[0]
        _expect("dout", dout, (T, self.n_out), y_rows.dtype)
        dy_rows, dweights = torch.empty_like(y_rows), torch.empty_like(weights)
        dlogits = torch.empty_like(logits)
        mlg.mlg_combine_backward(dout, y_rows, pos, weights, offsets[-1:], dy_rows, dweights, T,
                                 self.n_out, K, n)
        mlg.mlg_route_topk_backward(logits, indices, weights, dweights, dlogits, T,
                                    self.n_experts, K, self.renormalize)
        return dy_rows, dlogits

    def rows_backward(self, dx_rows):
        """The gradient of the last prefill()'s x, given that of its sorted rows."""
        pos = self._last()[4]
        n = pos.shape[0]
        _expect("dx_rows", dx_rows, (n, self.k_in))
        dx = torch.empty(n // self.top_k, self.k_in, dtype=dx_rows.dtype, device="cuda")
        mlg.mlg_combine(dx_rows, pos, None, dx, dx.shape[0], self.k_in, self.top_k, n)
        return dx

    def decode(self, x, logits, row_map):
        """The same for a decode batch, with the 4-bit weights."""
        codes, scales, zeros, group = self.q4
        row_map = self._batch(x, logits, row_map)
        x = x.contiguous()  # both products read its rows one after the other
        T, K, n = x.shape[0], self.top_k, x.shape[0] * self.top_k
        indices, weights = self.route(logits)
        rows = torch.empty(n, self.n_out, dtype=torch.bfloat16, device="cuda")
        out = torch.empty(T, self.n_out, dtype=torch.bfloat16, device="cuda")
        mlg.mlg_gather_q4(x, indices, codes, scales, zeros, rows, n, self.k_in, self.n_out, K,
                          self.n_experts, group)
        mlg.mlg_gather_bgmv(x, indices, row_map, self.a_table, self.b_table, self.scale_table,
                            rows, n, self.k_in, self.max_rank, self.n_out, K, self.n_experts)
        mlg.mlg_combine(rows, None, weights, out, T, self.n_out, K, n)
        return out


def random_projection(seed: int, n_experts: int, k_in: int, n_out: int, top_k: int, rank: int,
                      group: int) -> MoeProjection:
    """Random 4-bit experts, their bf16 form as the dense weights, and a pair for every second
    expert."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    shape = (n_experts, n_out, k_in // group)
    codes = torch.randint(0, 256, (n_experts, n_out, k_in // 2), generator=g, device="cuda",
                          dtype=torch.uint8)
    scales = ((torch.rand(shape, generator=g, device="cuda") + 0.5) / (4 * k_in ** 0.5)).to(
        torch.bfloat16)
    zeros = torch.randint(5, 11, shape, generator=g, device="cuda", dtype=torch.uint8)
    q = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).unflatten(-1, (-1, group)).float()
    dense = ((q - zeros[..., None].float()) * scales[..., None].float()).flatten(-2)
    ids = list(range(0, n_experts, 2))
    A = torch.randn(len(ids), rank, k_in, generator=g, device="cuda") / k_in ** 0.5
    B = torch.randn(len(ids), n_out, rank, generator=g, device="cuda") / rank ** 0.5
    scale = np.linspace(0.5, 2.0, len(ids)).astype(np.float32)
    return MoeProjection(dense.to(torch.bfloat16), top_k,
                         lora=(ids, A.to(torch.bfloat16), B.to(torch.bfloat16), scale),
                         q4=(codes, scales, zeros, group))


def main() -> None:
    p = random_projection(0, 128, 768, 2048, 8, 16, 64)
    for name, T, run in (("prefill", 4096, lambda x, l: p.prefill(x, l, keep=False)),
                         ("decode", 64, lambda x, l: p.decode(x, l, torch.zeros(
                             x.shape[0], dtype=torch.int32, device="cuda")))):
        x = torch.randn(T, p.k_in, device="cuda").to(torch.bfloat16)
        logits = torch.randn(T, p.n_experts, device="cuda").to(torch.bfloat16)
        for _ in range(3):
            run(x, logits)
        begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        begin.record()
        for _ in range(20):
            run(x, logits)
        end.record()
        torch.cuda.synchronize()
        print(f"{name}: {T} tokens, top {p.top_k} of {p.n_experts} experts, "
              f"{begin.elapsed_time(end) * 50:.1f} us")


if __name__ == "__main__":
    main()
