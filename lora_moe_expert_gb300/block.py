"""One MoE block of a decoder layer, from the residual stream to the residual stream, with its
experts' weights in 8-bit floating point.

``MoeBlock`` holds what a serving process keeps (the norms' weights, the router, the experts, the
LoRA tables) and runs a batch through

* any number of tokens: the norm before the block -> the router's logits (a library product) and
  top_k -> rows into expert order, in 8 bits -> the gate and up product (and its LoRA fold) -> the
  activation, in 8 bits again -> the down product (and its fold) -> the weighted sum of a token's
  rows -> the norm after the block, its gate, the residual sum and the norm before the next block;
* a few tokens without adapters: the same with the layer in one call, whose hidden states and
  activations are not brought to 8 bits (by several percent of the block's output another result);
* the gradients of the last step, for training the norms, the gate and what lies on either side of
  frozen experts.

torch provides device memory, streams and the router's product only.

    python -m lora_moe_expert_gb300.block     # runs both forms on random data
"""
from __future__ import annotations

import numpy as np
import torch

import lora_moe_expert_gb300 as mlg
from lora_moe_expert_gb300.projection import _expect, _i32

F8 = torch.float8_e4m3fn


def _blocks(n: int) -> int:
    return -(-n // mlg.MLG_F8_BLOCK)


def _new(*shape, dtype=torch.bfloat16):
    return torch.empty(*shape, dtype=dtype, device="cuda")


def quantize_weights(w):
    """[n_experts, n, k] weights as (codes, scales): e4m3 with a scale for each 128 x 128 block, the
    block's largest magnitude over 448 (once, when weights are loaded)."""
    E, n, k = w.shape
    B = mlg.MLG_F8_BLOCK
    codes = torch.empty(E, n, k, dtype=F8, device=w.device)
    scales = torch.empty(E, _blocks(n), _blocks(k), dtype=torch.float32, device=w.device)
    for e in range(E):
        padded = torch.zeros(_blocks(n) * B, _blocks(k) * B, device=w.device)
        padded[:n, :k] = w[e]
        tiles = padded.view(_blocks(n), B, _blocks(k), B)
        scales[e] = (tiles.abs().amax((1, 3)) / 448).clamp(min=2.0 ** -126)
        tiles /= scales[e][:, None, :, None]
        codes[e] = padded[:n, :k].clamp(-448, 448).to(F8)
    return codes, scales


class _Lora:
    """The tables of one projection's pairs: (ids, A [n, max_rank, k_in], B [n, n_out, max_rank],
    scale)."""

    def __init__(self, pairs, n_experts: int, k_in: int, n_out: int):
        ids, A, B, scale = pairs
        self.A, self.B = A.contiguous(), B.contiguous()
        self.max_rank = A.shape[1]
        _expect("A", self.A, (len(ids), self.max_rank, k_in), torch.bfloat16)
        _expect("B", self.B, (len(ids), n_out, self.max_rank), torch.bfloat16)
        at = [[t.data_ptr() + i * t[0].numel() * 2 for i in range(len(ids))]
              for t in (self.A, self.B)]
        a, b, s = (np.zeros(n_experts, t) for t in (np.uint64, np.uint64, np.float32))
        pa, pb, ps = mlg.mlg_pack_expert_tables(ids, *at, scale)
        a[:pa.size], b[:pb.size], s[:ps.size] = pa, pb, ps
        self.tables = _new(n_experts, dtype=torch.int64), _new(n_experts, dtype=torch.int64), \
            _new(n_experts, dtype=torch.float32)
        mlg.mlg_upload_expert_tables(a, b, s, *self.tables)


class MoeBlock:
    """norm_in [hidden] and norm_out [hidden] (or None) bf16: the norms before and after the block;
    router [n_experts, hidden] bf16; gate_up ([n_experts, 2 inter, hidden] codes, scales) and down
    ([n_experts, hidden, inter] codes, scales) as quantize_weights gives them; lora_gate_up, lora_down:
    pairs of the adapted experts as of MoeProjection, or None.

    few_tokens: batches of up to as many tokens take the layer in one call, where the block has no
    adapter.  With 0 every batch goes call by call: then a token's rows are the same alone and in any
    batch, and an adapter changes the tokens that use it alone."""

    def __init__(self, norm_in, router, gate_up, down, top_k: int, norm_out=None,
                 lora_gate_up=None, lora_down=None, renormalize: bool = True,
                 residual_scale: float = 1.0, branch_scale: float = 1.0, eps: float = 1e-6,
                 few_tokens: int = mlg.MLG_MOE_MAX_TOKENS):
        if not 0 <= few_tokens <= mlg.MLG_MOE_MAX_TOKENS:
            raise ValueError(f"few_tokens: 0 to {mlg.MLG_MOE_MAX_TOKENS} expected, {few_tokens} given")
        self.few_tokens = few_tokens
        self.gate_up, self.gate_up_scales = (t.contiguous() for t in gate_up)
        self.down, self.down_scales = (t.contiguous() for t in down)
        E, H, inter = self.down.shape
        self.n_experts, self.hidden, self.inter, self.top_k = E, H, inter, top_k
        _expect("gate_up", self.gate_up, (E, 2 * inter, H), F8)
        _expect("down", self.down, (E, H, inter), F8)
        _expect("gate_up_scales", self.gate_up_scales, (E, _blocks(2 * inter), _blocks(H)),
                torch.float32)
        _expect("down_scales", self.down_scales, (E, _blocks(H), _blocks(inter)), torch.float32)
        _expect("norm_in", norm_in, (H,), torch.bfloat16)
        _expect("router", router, (E, H), torch.bfloat16)
        if norm_out is not None:
            _expect("norm_out", norm_out, (H,), torch.bfloat16)
        self.norm_in, self.norm_out, self.router = norm_in, norm_out, router
        self.lora_gate_up = lora_gate_up and _Lora(lora_gate_up, E, H, 2 * inter)
        self.lora_down = lora_down and _Lora(lora_down, E, inter, H)
        self.renormalize, self.eps = renormalize, eps
        self.residual_scale, self.branch_scale, self.saved = residual_scale, branch_scale, None

    def forward(self, x, gate=None, row_map=None, next_norm=None, z=None, keep: bool = False):
        """x [tokens, hidden] bf16 -> (out, z): the residual stream after the block, and its norm with
        the weight next_norm [hidden] (None: z is None).  gate [tokens, 1 or hidden] scales the
        block's output; row_map [tokens] int32, negative for a token without adapter (None: with
        the adapters that there are, all tokens); z, the norm of x, where the block before has
        computed it.  With keep, self.saved holds what was computed (x, gate and out themselves, not
        copies), for backward(), until the next forward(): one batch at a time.  Without, nothing is
        held, also of a step before."""
        T, H = x.shape[0], self.hidden
        _expect("x", x, (T, H), torch.bfloat16)
        if row_map is not None:
            _expect("row_map", row_map, (T,), torch.int32)
            row_map = row_map.contiguous()
        if gate is not None:
            _expect("gate", gate, (T, H if gate.shape[-1] == H else 1), torch.bfloat16)
        if next_norm is not None:
            _expect("next_norm", next_norm, (H,), torch.bfloat16)
        s = {"x": x, "gate": gate, "z": z, "next_norm": next_norm}
        if z is None:
            s["z"] = _new(T, H)
            mlg.mlg_block_norm(x, None, None, None, self.norm_in, None, s["z"], T, H, eps=self.eps)
        else:
            _expect("z", z, (T, H), torch.bfloat16)
        s["logits"] = s["z"] @ self.router.t()
        s["indices"] = _i32(T, self.top_k)
        s["weights"] = _new(T, self.top_k, dtype=torch.float32)
        adapted = self.lora_gate_up is not None or self.lora_down is not None
        if T <= self.few_tokens and not adapted:
            self._layer(s, T)
        else:
            self._rows(s, T, row_map)
        out, z_next = _new(T, H), None if next_norm is None else _new(T, H)
        mlg.mlg_block_norm(x, s["y"], gate, self.norm_out, next_norm, out, z_next, T, H,
                           self.residual_scale, self.branch_scale, self.eps)
        s["out"] = out
        self.saved = s if keep else None
        return out, z_next

    def _layer(self, s, T):
        """The layer in one call; its activations are in a form of its own and are not saved."""
        act, s["y"] = _new(T * self.top_k, self.inter), _new(T, self.hidden)
        mlg.mlg_moe_layer_f8(s["logits"], s["z"].contiguous(), self.gate_up, self.gate_up_scales,
                             self.down, self.down_scales, s["indices"], s["weights"], act, s["y"],
                             T, self.hidden, self.inter, self.n_experts, self.top_k,
                             self.renormalize)

    def _rows(self, s, T, row_map):
        """The layer call by call, over the (token, slot) rows in expert order."""
        E, K, H, inter, n = self.n_experts, self.top_k, self.hidden, self.inter, T * self.top_k
        mlg.mlg_route_topk(s["logits"], s["indices"], s["weights"], T, E, K, self.renormalize)
        s["offsets"], s["src"], s["pos"] = _i32(E + 1), _i32(n), _i32(n)
        mlg.mlg_sort_slots(s["indices"], None, s["offsets"], s["src"], s["pos"], n, K, E)
        s["q"], s["scales"] = _new(n, H, dtype=F8), _new(n, _blocks(H), dtype=torch.float32)
        mlg.mlg_rows_f8(s["z"], s["pos"], s["q"], s["scales"], T, H, K, n)
        s["gate_up"] = _new(n, 2 * inter)
        mlg.mlg_grouped_gemm_f8(s["q"], s["scales"], s["offsets"], self.gate_up,
                                self.gate_up_scales, s["gate_up"], n, H, 2 * inter, E)
        if self.lora_gate_up is not None and n > 0:
            mlg.mlg_grouped_down_all_windows(
                s["z"].contiguous(), s["offsets"], s["src"], row_map, *self.lora_gate_up.tables,
                s["gate_up"], H, self.lora_gate_up.max_rank, 2 * inter, K, E, n, n)
        s["act"] = None if self.lora_down is None else _new(n, inter)
        s["act_q"], s["act_scales"] = _new(n, inter, dtype=F8), _new(n, _blocks(inter),
                                                                     dtype=torch.float32)
        mlg.mlg_swiglu_f8(s["gate_up"], s["act"], s["act_q"], s["act_scales"], n, inter)
        s["rows"] = _new(n, H)
        mlg.mlg_grouped_gemm_f8(s["act_q"], s["act_scales"], s["offsets"], self.down,
                                self.down_scales, s["rows"], n, inter, H, E)
        if self.lora_down is not None and n > 0:
            mlg.mlg_grouped_down_xrows(s["act"], s["offsets"], s["src"], row_map,
                                       *self.lora_down.tables, s["rows"], inter,
                                       self.lora_down.max_rank, H, K, E, 0, n, n)
        s["y"] = _new(T, H)
        mlg.mlg_combine(s["rows"], s["pos"], s["weights"], s["y"], T, H, K, n)

    def backward(self, dout, dz=None):
        """The gradients of the last forward(), one with keep, given those of out (or None) and of z:
        {"x": of the residual stream past the block, "y": of the layer's output, "gate", "norm_out",
        "next_norm"} (the last three where they are there; the weights' are fp32)."""
        if self.saved is None:
            raise RuntimeError("the last forward() was not one with keep")
        s, (T, H) = self.saved, self.saved["x"].shape
        if (s["next_norm"] is None) != (dz is None):
            raise ValueError("dz: the gradient of forward()'s z expected, where it returned one")
        for what, t in (("dout", dout), ("dz", dz)):
            if t is not None:
                _expect(what, t, (T, H), torch.bfloat16)
        got = {"x": _new(T, H), "y": _new(T, H)}
        if s["gate"] is not None:
            got["gate"] = torch.empty_like(s["gate"])
        for name, w in (("norm_out", self.norm_out), ("next_norm", s["next_norm"])):
            if w is not None:
                got[name] = _new(H, dtype=torch.float32)
        partial = _new(2 * mlg.MLG_NORM_PARTIALS * H, dtype=torch.float32)
        mlg.mlg_block_norm_backward(dout, dz, s["out"], s["y"], s["gate"], self.norm_out,
                                    s["next_norm"], got["x"], got["y"], got.get("gate"),
                                    got.get("norm_out"), got.get("next_norm"), partial, T, H,
                                    self.residual_scale, self.branch_scale, self.eps)
        return got


def random_block(seed: int, n_experts: int, hidden: int, inter: int, top_k: int, rank: int = 0,
                 **options) -> MoeBlock:
    """Random weights, and with a rank pairs for every second expert."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def weights(*shape, by):
        return torch.randn(*shape, generator=g, device="cuda") / by

    def pairs(k, n):
        ids = list(range(0, n_experts, 2))
        return (ids, weights(len(ids), rank, k, by=k ** 0.5).to(torch.bfloat16),
                weights(len(ids), n, rank, by=rank ** 0.5).to(torch.bfloat16),
                np.linspace(0.5, 2.0, len(ids)).astype(np.float32))

    norm = lambda: (weights(hidden, by=8) + 1).to(torch.bfloat16)  # noqa: E731
    lora = dict(lora_gate_up=pairs(hidden, 2 * inter), lora_down=pairs(inter, hidden)) if rank else {}
    return MoeBlock(norm(), weights(n_experts, hidden, by=hidden ** 0.5).to(torch.bfloat16),
                    quantize_weights(weights(n_experts, 2 * inter, hidden, by=hidden ** 0.5)),
                    quantize_weights(weights(n_experts, hidden, inter, by=inter ** 0.5)), top_k,
                    norm_out=norm(), **lora, **options)


def main() -> None:
    block = random_block(0, 128, 2048, 768, 8)
    next_norm = torch.ones(2048, dtype=torch.bfloat16, device="cuda")
    for T in (1, 16, 64, 4096):
        x = torch.randn(T, 2048, device="cuda").to(torch.bfloat16)
        for _ in range(3):
            block.forward(x, next_norm=next_norm)
        begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        begin.record()
        for _ in range(20):
            block.forward(x, next_norm=next_norm)
        end.record()
        torch.cuda.synchronize()
        print(f"{T} tokens, top {block.top_k} of {block.n_experts} experts, "
              f"{begin.elapsed_time(end) * 50:.1f} us")


if __name__ == "__main__":
    main()
