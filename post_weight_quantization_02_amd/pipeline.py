"""Whole-model quantization around the layer solver.

itwiki "GPTQ", section "최소 구현" (the paragraph after the sketch): the model is
processed one transformer block at a time, front to back; the calibration inputs
are run through the block while H is accumulated for each of its layers, the
layers are quantized, and the quantized block's outputs become the next block's
inputs.  molayo1419.me (nanoGPT post), section 3: forward hooks capture the inputs
of every nn.Linear and each layer is quantized independently -- the
``sequential=False`` mode here (every block sees the unquantized model's
activations).

Per block: one pass of every calibration batch with forward pre-hooks on the
block's nn.Linear layers, each hook adding 2 X^T X of that layer's input rows to
the layer's H on the device (gptq_hessian_accumulate -- the activations are never
stored); then for each layer the damped factor and the lazy-batch loop (or their
act-order forms), and What written back into the layer's weight
(gptq_dequantize); then, in sequential mode, a second pass with the quantized
weights whose outputs are the next block's inputs.  Every quantizer step runs in
the library's kernels on the current stream; the forward passes are the caller's
model.  Biases are left as they are.

Beside it, without calibration: ``quantize_model_fp8`` puts an ``Fp8Linear`` in the place
of every nn.Linear (e4m3 weights in 128 x 128 tiles, inputs quantized per row on every
call).  ``evaluate`` scores a model, quantized or not, on given texts: mean negative log
probability and perplexity (the pages' loss and perplexity before and after), entropy,
and how often the given token was the most probable one.
"""
from __future__ import annotations

import dataclasses
import math
from typing import Dict, List, Optional, Sequence

import torch as _t

from . import (NotPositiveDefinite, _torch, gptq_act_order_perm, gptq_dequantize, gptq_fp8_matmul, gptq_fp8_quantize,
               gptq_hessian_accumulate, gptq_prepare_hinv, gptq_prepare_hinv_perm, gptq_quantize_layer,
               gptq_quantize_layer_perm, gptq_token_logprobs)


@dataclasses.dataclass
class LayerQuant:
    codes: object            # uint8 [out x in], original column order
    scales: object           # fp32 [out x n_groups]
    zeros: object            # int32 [out x n_groups]
    err: object              # fp64 [1]: ||X (W0 - What)^T||^2 over the layer's calibration rows
    lam: object              # fp32 [1]
    perm: object = None      # act-order: the quantization order
    g_idx: object = None     # act-order: column -> group
    H: object = None         # the layer's H (kept on request)


@dataclasses.dataclass
class BlockQuant:
    layers: Dict[str, LayerQuant]
    inputs: Optional[List[object]] = None   # the block's calibration inputs (kept on request)


def linear_layers(block) -> List:
    """(name, module) of every nn.Linear in the block, in registration order."""
    torch = _torch()
    return [(n, m) for n, m in block.named_modules() if isinstance(m, torch.nn.Linear)]


def quantize_model(blocks: Sequence, x_batches: Sequence, bits: int, group_size: int = 0,
                   block_size: int = 128, percdamp: float = 0.01, act_order: bool = False,
                   sequential: bool = True, keep_inputs: bool = False, keep_hessians: bool = False,
                   stream=None):
    """Quantize every nn.Linear of ``blocks`` (torch modules on the GPU, each mapping
    a batch to the next block's input), front to back, with ``x_batches`` (device
    tensors) as the first block's calibration inputs.  The layers' weights are
    replaced by What in place.  Returns (per-block results, the last block's
    outputs for the batches).  Raises NotPositiveDefinite if a layer's damped H
    could not be factored (checked once per block, before any weight of that
    block is replaced, so the block's weights are then left as they were)."""
    torch = _torch()
    xs = list(x_batches)
    results = []
    with torch.no_grad():
        for block in blocks:
            lins = linear_layers(block)
            Hs = {n: torch.zeros(m.in_features, m.in_features, dtype=torch.float32, device=m.weight.device)
                  for n, m in lins}

            def hook_for(name, width):
                def hook(_mod, inp):
                    x = inp[0].reshape(-1, width)
                    gptq_hessian_accumulate(Hs[name], x if x.is_contiguous() else x.contiguous(), stream=stream)
                return hook

            handles = [m.register_forward_pre_hook(hook_for(n, m.in_features)) for n, m in lins]
            ys = []                    # the unquantized block's outputs, kept for independent mode
            try:
                for x in xs:
                    y = block(x)
                    if not sequential:
                        ys.append(y)
            finally:
                for h in handles:
                    h.remove()
            layers, infos = {}, []
            for n, m in lins:
                W0 = m.weight.data
                if act_order:
                    perm = gptq_act_order_perm(Hs[n], stream=stream)
                    U, lam, info = gptq_prepare_hinv_perm(Hs[n], perm, percdamp, stream=stream)
                    codes, scales, zeros, g_idx, err = gptq_quantize_layer_perm(
                        W0, U, lam, perm, bits, group_size, block_size, stream=stream)
                else:
                    perm = g_idx = None
                    U, lam, info = gptq_prepare_hinv(Hs[n], percdamp, stream=stream)
                    codes, scales, zeros, err = gptq_quantize_layer(W0, U, lam, bits, group_size, block_size,
                                                                    stream=stream)
                # What goes to a staging tensor: the weights are replaced only once every
                # layer of the block is known to have been factored (U is unspecified
                # when info != 0, and a caller may catch the error and retry)
                w_hat = gptq_dequantize(codes, scales, zeros, group_size, g_idx, out_dtype=W0.dtype,
                                        stream=stream)
                layers[n] = LayerQuant(codes, scales, zeros, err, lam, perm, g_idx, Hs[n] if keep_hessians else None)
                infos.append((n, info, W0, w_hat))
            (stream or torch.cuda.current_stream()).synchronize()
            for n, info, _, _ in infos:
                if int(info.item()) != 0:
                    raise NotPositiveDefinite(int(info.item()))
            for _, _, W0, w_hat in infos:
                W0.copy_(w_hat)
            results.append(BlockQuant(layers, xs if keep_inputs else None))
            xs = [block(x) for x in xs] if sequential else ys
    return results, xs


def _own_rows(t):
    """t [rows x width], copied unless its columns are adjacent and its rows do not overlap."""
    if t.stride(1) == 1 and (t.shape[0] < 2 or t.stride(0) >= t.shape[1]):
        return t
    return t.clone(memory_format=_t.contiguous_format)


class Fp8Linear(_t.nn.Module):
    """A linear layer with e4m3 weights: y = dequantized(x) dequantized(W)^T + bias in
    x's dtype (fp32, fp16 or bf16; with fp32 the sums are fp32 too, see gptq_fp8_matmul),
    x's rows quantized on every call.  For inference: inputs that ask for a gradient are
    refused."""

    def __init__(self, weight, bias=None):
        super().__init__()
        self.out_features, self.in_features = weight.shape
        codes, scales = gptq_fp8_quantize(_own_rows(weight.detach()), 128)
        self.register_buffer("codes", codes.view(_t.uint8))      # bit patterns: a cast of the model leaves them alone
        self.register_buffer("scales", scales)
        self.register_buffer("bias", None if bias is None else bias.detach().clone())

    def _apply(self, fn, recurse=True):
        scales = self.scales
        super()._apply(fn, recurse)
        if self.scales.dtype != scales.dtype:       # model.half() and the like: the scales stay fp32
            self.scales = scales.to(self.scales.device)
        self._align_rows()
        return self

    def _load_from_state_dict(self, *args, **kwargs):
        super()._load_from_state_dict(*args, **kwargs)
        self._align_rows()

    def _align_rows(self):
        """Rows of codes a multiple of 128 bytes apart again, which the product's fast kernels
        want: a move to another device and some ways of loading close the gaps."""
        n, k = self.codes.shape
        if self.codes.stride(0) % 16 or self.codes.stride(1) != 1:
            codes = self.codes.new_zeros(n, (k + 127) // 128 * 128)[:, :k]
            self.codes = codes.copy_(self.codes)

    def forward(self, x):
        if x.requires_grad and _t.is_grad_enabled():
            raise ValueError("Fp8Linear has no backward pass: detach its input or call it under torch.no_grad()")
        codes, scales = gptq_fp8_quantize(_own_rows(x.reshape(-1, self.in_features)))
        bias = self.bias if self.bias is None or self.bias.dtype == x.dtype else self.bias.to(x.dtype)
        y = gptq_fp8_matmul(codes, scales, self.codes, self.scales, bias, out_dtype=x.dtype)
        return y.reshape(*x.shape[:-1], self.out_features)

    def extra_repr(self) -> str:
        return f"in_features={self.in_features}, out_features={self.out_features}, bias={self.bias is not None}"


def _in_place_of(child):
    """The Fp8Linear of a Linear, with its mode and its forward hooks: the same tables, so a
    hook's handle still removes it.  Backward hooks have nothing to wait for."""
    layer = Fp8Linear(child.weight, child.bias)
    layer.training = child.training
    for table in ("_forward_pre_hooks", "_forward_pre_hooks_with_kwargs", "_forward_hooks",
                  "_forward_hooks_with_kwargs", "_forward_hooks_always_called"):
        setattr(layer, table, getattr(child, table))
    return layer


def quantize_model_fp8(blocks: Sequence) -> List[List[str]]:
    """Put an Fp8Linear in the place of every nn.Linear of ``blocks`` (torch modules on
    the GPU), in place.  A layer used under several names stays one layer.  Subclasses of
    nn.Linear stay as they are (nn.MultiheadAttention reads its output projection's weight
    itself), and so do layers whose weight or bias is no parameter of their own but computed on
    every call (weight_norm, prune).  A layer's mode and forward hooks move to its Fp8Linear.  All
    layers are coded before the first one is replaced.  Returns the names of the replaced
    layers, block by block."""
    names, made, places = [], {}, []
    for block in blocks:
        if isinstance(block, _t.nn.Linear):
            raise ValueError("a block that is itself a Linear cannot be replaced in place: use Fp8Linear")
        names.append([])
        for parent_name, parent in list(block.named_modules()):
            for name, child in list(parent._modules.items()):     # under every name, a shared layer's too
                if type(child) is _t.nn.Linear and {"weight", "bias"} <= child._parameters.keys():
                    if id(child) not in made:
                        made[id(child)] = _in_place_of(child)
                    places.append((parent, name, made[id(child)]))
                    names[-1].append(f"{parent_name}.{name}" if parent_name else name)
    for parent, name, layer in places:
        setattr(parent, name, layer)
    return names


@dataclasses.dataclass
class Evaluation:
    tokens: int              # scored positions (those with a token >= 0)
    nll: float               # mean negative log probability of the given tokens, in nats
    perplexity: float        # e^nll
    entropy: float           # mean entropy of the model's distributions there, in nats
    accuracy: float          # share of positions whose most probable token is the given one


def evaluate(blocks: Sequence, head, x_batches: Sequence, token_batches: Sequence,
             rows_per_call: int = 8192) -> Evaluation:
    """Score a model on given texts.  ``blocks`` map each batch of ``x_batches`` [S x T x d]
    on, ``head`` (an nn.Linear, an Fp8Linear, any module) maps hidden rows [rows x d] to
    logits [rows x v] (fp32, fp16 or bf16); ``token_batches`` hold the tokens to be
    predicted there, int64 [S x T], negative where there is none (padding, a text's last
    position).  The head and the scores run on at most ``rows_per_call`` rows at a time.  The
    modules run in the mode they are in: call eval() on those with dropout first.  The device
    is waited for once, at the end."""
    if len(x_batches) != len(token_batches):
        raise ValueError("x_batches and token_batches differ in number")
    if rows_per_call < 1:
        raise ValueError("rows_per_call must be at least 1")
    sums, width = None, 0
    with _t.no_grad():
        for x, tokens in zip(x_batches, token_batches):
            if tokens.shape != x.shape[:-1]:
                raise ValueError(f"tokens of shape {tuple(tokens.shape)} for a batch of shape {tuple(x.shape)}")
            for block in blocks:
                x = block(x)
            hidden, tok = x.reshape(-1, x.shape[-1]), tokens.reshape(-1).contiguous()
            if sums is None:
                sums = _t.zeros(5, dtype=_t.float64, device=x.device)
            for i in range(0, hidden.shape[0], rows_per_call):
                t = tok[i:i + rows_per_call]
                logits = head(hidden[i:i + rows_per_call])
                width = logits.shape[1]
                lp, entropy, ids, _ = gptq_token_logprobs(logits, t, 1)
                scored = t >= 0
                sums += _t.stack([scored.sum().double(), lp.double().sum(),
                                  entropy.double().masked_fill(~scored, 0.0).sum(),
                                  ((ids[:, 0] == t) & scored).sum().double(),
                                  (t >= width).sum().double()])       # scored as NaN, refused below
    n, lp, entropy, hits, above = [0.0] * 5 if sums is None else sums.tolist()
    if above > 0:
        raise ValueError(f"a token is not below the {width} logits")
    if n == 0:
        raise ValueError("no position holds a token to be scored")
    nll = -lp / n
    return Evaluation(int(n), nll, math.inf if nll >= 700 else math.exp(nll), entropy / n, hits / n)
