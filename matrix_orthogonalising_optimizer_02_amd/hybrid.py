"""Hybrid optimizer: Muon for the 2-D weights inside transformer blocks, AdamW for the rest.

"Scaling Muon for Diffusion Transformers" (setup paragraph) applies Muon only to the
2-D weights of the transformer blocks, about 99% of the trainable parameters, and keeps
biases, normalisation parameters and every parameter outside the blocks on an
auxiliary AdamW group (lr 1e-4). "Muon is Scalable for LLM Training" (Sec. 2.2,
matching-update-RMS paragraph) pairs the two the same way and lets them share the
weight decay. Both halves run in libmuon_rocm.so: muon_step for the Muon group (one
launch sequence per step for all of its matrices) and adamw_step for the AdamW group.

`dit_parameter_list` names and shapes the parameters of a double-stream (image and
text) diffusion transformer, whose block matrices are the pages' DiT shapes: qkv
[3H, H], proj [H, H], MLP up [4H, H] and down [H, 4H], adaLN modulation [6H, H].
"""
from __future__ import annotations

from typing import Dict, List, Optional, Sequence, Tuple

from . import binding as B
from .multi import AdamWMulti, GradNorm

BLOCK_PREFIX = "blocks."

# Scales of the pages' model family (1.3B, 4B, 9B, 15B), read as hidden size and depth
# of a double-stream backbone whose block holds 2 x 18 H^2 matrix weights.
DIT_SCALES = {
    "1.3B": (2048, 9),
    "4B": (3072, 12),
    "9B": (4096, 15),
    "15B": (5120, 16),
}


def goes_to_muon(name: str, shape: Sequence[int]) -> bool:
    """2-D parameters inside a transformer block go to Muon; everything else to AdamW."""
    return len(shape) == 2 and name.startswith(BLOCK_PREFIX)


def split_param_groups(named_shapes) -> Tuple[List[str], List[str]]:
    """(Muon names, AdamW names) for an iterable of (name, shape), order preserved."""
    muon, adamw = [], []
    for name, shape in named_shapes:
        (muon if goes_to_muon(name, tuple(shape)) else adamw).append(name)
    return muon, adamw


def dit_parameter_list(hidden: int, depth: int, head_dim: int = 128, latent_channels: int = 16,
                       patch: int = 2, text_dim: int = 4096, pooled_dim: int = 2048,
                       freq_dim: int = 256) -> List[Tuple[str, Tuple[int, ...]]]:
    """(name, shape) of every trainable parameter of a double-stream DiT.

    Per block and stream: attention qkv and output projection, q/k RMSNorm weights,
    a 4x MLP and the adaLN modulation, each linear with a bias. Outside the blocks:
    patch and text embedders, the timestep and pooled-text embedders, and the final
    adaLN + projection layer (latent channels x patch^2 outputs).
    """
    h = hidden
    out_dim = latent_channels * patch * patch
    params: List[Tuple[str, Tuple[int, ...]]] = []

    def linear(name, rows, cols):
        params.append((f"{name}.weight", (rows, cols)))
        params.append((f"{name}.bias", (rows,)))

    linear("x_embedder", h, out_dim)
    linear("context_embedder", h, text_dim)
    linear("time_embed.fc1", h, freq_dim)
    linear("time_embed.fc2", h, h)
    linear("pooled_embed.fc1", h, pooled_dim)
    for i in range(depth):
        for stream in ("img", "txt"):
            p = f"{BLOCK_PREFIX}{i}.{stream}"
            linear(f"{p}.attn.qkv", 3 * h, h)
            params.append((f"{p}.attn.q_norm.weight", (head_dim,)))
            params.append((f"{p}.attn.k_norm.weight", (head_dim,)))
            linear(f"{p}.attn.proj", h, h)
            linear(f"{p}.mlp.up", 4 * h, h)
            linear(f"{p}.mlp.down", h, 4 * h)
            linear(f"{p}.mod", 6 * h, h)
    linear("final_layer.mod", 2 * h, h)
    linear("final_layer.linear", out_dim, h)
    return params


def count_params(named_shapes) -> Tuple[int, int]:
    """(Muon elements, AdamW elements)."""
    mu = ad = 0
    for name, shape in named_shapes:
        n = 1
        for d in shape:
            n *= int(d)
        if goes_to_muon(name, tuple(shape)):
            mu += n
        else:
            ad += n
    return mu, ad


class HybridOptimizer:
    """Periodic Row-wise Muon on the block matrices plus AdamW on the other parameters.

    named_params: mapping name -> fp32 CUDA tensor (contiguous). step(grads) takes a
    mapping with the same names and advances every parameter by one step; both groups
    share the 0-based step counter (Muon's refresh schedule, AdamW's bias correction).

    adamw_state_bits: None for adamw_step (fp32 moments, one launch for every 48 tensors);
    32 or 8 for AdamWMulti, one launch whatever their number, with moments of that width
    (8: a quarter of the memory, rounded stochastically from `seed`). AdamW's gradients
    may then be bfloat16 or float16 too, Muon's stay fp32.
    max_grad_norm: clip all gradients together to this l2 norm (needs 32 or 8 above). The
    factor stays on the device: Muon's gradients are scaled in place, AdamW's where they
    are read. `grad_norm` then holds the last step's norm and factor (float32 [2]).

    With adamw_state_bits no gradient is kept after the step that it was given to; who
    captures a step into a graph keeps its gradients for the replays.
    """

    def __init__(self, named_params: Dict[str, "object"], muon_hp: Optional[B.MuonHParams] = None,
                 adamw_hp: Optional[B.AdamWHParams] = None, adamw_state_bits: Optional[int] = None,
                 max_grad_norm: Optional[float] = None, seed: int = 0):
        import torch
        if adamw_state_bits not in (None, 8, 32):
            raise ValueError("adamw_state_bits must be None, 8 or 32")
        if max_grad_norm is not None and adamw_state_bits is None:
            raise ValueError("max_grad_norm needs adamw_state_bits 8 or 32")
        if max_grad_norm is not None and not 0.0 < max_grad_norm < float("inf"):
            raise ValueError("max_grad_norm must be finite and > 0")
        self.names = list(named_params)
        shapes = [(n, tuple(named_params[n].shape)) for n in self.names]
        self.muon_names, self.adamw_names = split_param_groups(shapes)
        self.params = named_params
        self.muon_hp = muon_hp or B.default_hparams()
        self.adamw_hp = adamw_hp or B.adamw_default_hparams()
        self.adamw_state_bits, self.max_grad_norm, self.seed = adamw_state_bits, max_grad_norm, seed
        self.momenta = {n: torch.zeros_like(named_params[n]) for n in self.muon_names}
        small = adamw_state_bits is not None
        self.exp_avg = {} if small else {n: torch.zeros_like(named_params[n]) for n in self.adamw_names}
        self.exp_avg_sq = {} if small else {n: torch.zeros_like(named_params[n]) for n in self.adamw_names}
        dev = next(iter(named_params.values())).device if named_params else "cuda"
        self.workspace = B.make_workspace([tuple(named_params[n].shape) for n in self.muon_names], dev) \
            if self.muon_names else None
        self._adamw = None  # descriptor array, built at the first step
        if small and self.adamw_names:
            self._adamw = AdamWMulti([named_params[n] for n in self.adamw_names], None, self.adamw_hp, adamw_state_bits,
                                     seed=seed)
        self._norm = self._muon_norm = None
        self.grad_norm = None
        self.step_count = 0

    def step(self, grads: Dict[str, "object"], stream=None, update_rms=None, counter=None, lr=None):
        """One step. What either half refuses is refused before anything is written: weights,
        states, gradients and step_count are then as they were.

        counter, lr: AdamW's step number and learning rate on the device (AdamWMulti.step), for
        steps that are captured into a graph. With the host's step_count a replay would repeat
        the bias corrections of the captured step and, with 8-bit states, its rounding bits, and
        rounding would no longer be unbiased. Every run of the step increases the counter (it is
        left alone where AdamW has no elements).
        Muon's schedule stays the host's: capture a whole cycle of period_k steps (or a graph for
        each kind of step), and set step_count by the counter before state_dict()."""
        if counter is not None and self.adamw_state_bits is None:
            raise ValueError("a counter needs adamw_state_bits 8 or 32")
        if counter is not None and not isinstance(counter, B._torch().Tensor):
            raise ValueError("a counter is a tensor on the device; otherwise set step_count")
        if counter is None and lr is not None:
            raise ValueError("lr as a tensor goes with a counter; otherwise set adamw_hp.lr")
        gm, ga = [grads[n] for n in self.muon_names], [grads[n] for n in self.adamw_names]
        at, factor = self.step_count if counter is None else counter, None
        try:
            if self.adamw_names:
                self._check_adamw(ga, stream, at, lr)
            # muon_step checks all of its arguments before its first launch
            muon = B.MuonCall([self.params[n] for n in self.muon_names], [self.momenta[n] for n in self.muon_names], gm,
                              self.step_count, self.muon_hp, self.workspace, stream, update_rms) if gm else None
            if self.max_grad_norm is not None and self.names:
                if gm:
                    muon.check()
                factor = self._clip([grads[n] for n in self.names], gm, stream)
            if gm:
                muon.run()
            if self.adamw_names and self.adamw_state_bits is None:
                self._adamw.step(self.step_count, stream)
            elif self.adamw_names:
                self._adamw.step(at, factor, stream, None, lr)
        finally:
            if self.adamw_state_bits is not None:
                for held in (self._adamw, self._norm, self._muon_norm):
                    if held is not None:
                        held.release_grads()
        self.step_count += 1

    def _check_adamw(self, g, stream, at, lr):
        """Gives AdamW its gradients; all that its step refuses is refused here."""
        if self.adamw_state_bits is not None:
            self._adamw.set_grads(g, stream)
            self._adamw.check_step(at, lr)
            return
        if self._adamw is None:
            self._adamw = B.AdamWGroup([self.params[n] for n in self.adamw_names], g,
                                       [self.exp_avg[n] for n in self.adamw_names],
                                       [self.exp_avg_sq[n] for n in self.adamw_names], self.adamw_hp)
        elif not all(a is b for a, b in zip(g, self._adamw.tensors[1])):
            self._adamw.set_grads(g)
        self._adamw.check_step(at)

    def _clip(self, g, gm, stream):
        """Measures all gradients, scales Muon's; the factor for AdamW's (device tensor)."""
        if self._norm is None:
            norm = GradNorm(g, stream)
            self._muon_norm = GradNorm(gm, stream) if gm else None
            self._norm = norm
        else:
            self._norm.set_grads(g, stream)
            if gm:
                self._muon_norm.set_grads(gm, stream)
        self.grad_norm, _ = self._norm.measure(self.max_grad_norm, stream)
        if gm:
            self._muon_norm.scale_(self._norm.factor, stream)
        return self._norm.factor

    def state_dict(self):
        state = {"step": self.step_count, "momenta": {n: t.clone() for n, t in self.momenta.items()}}
        if self.adamw_state_bits is None:
            state["exp_avg"] = {n: t.clone() for n, t in self.exp_avg.items()}
            state["exp_avg_sq"] = {n: t.clone() for n, t in self.exp_avg_sq.items()}
        elif self._adamw is None:
            state["adamw"] = None
        else:
            state["adamw"] = {"names": list(self.adamw_names), **self._adamw.state_dict()}
        return state

    def load_state_dict(self, state):
        """The saved states, by parameter name; nothing is changed where one does not fit. The
        rounding bits of 8-bit states go by an AdamW parameter's position in this optimizer."""
        if (self.adamw_state_bits is None) != ("exp_avg" in state):
            raise ValueError("the saved AdamW states are of another kind than this optimizer's")
        step = int(state["step"])
        groups = [("momenta", self.momenta), ("exp_avg", self.exp_avg), ("exp_avg_sq", self.exp_avg_sq)]
        for key, dst in groups:
            for n, t in dst.items():
                if state[key][n].shape != t.shape:
                    raise ValueError(f"{key} of {n} has another shape")
        if self.adamw_state_bits is not None and self._adamw is not None:
            self._adamw.load_state_dict(self._by_name(state["adamw"]))  # checks all before it copies
        self.step_count = step
        for key, dst in groups:
            for n, t in dst.items():
                t.copy_(state[key][n])

    def _by_name(self, saved):
        """AdamW's saved lists in this optimizer's order. Without names (as an earlier version
        saved them) they are in that order already."""
        if saved is None:
            raise ValueError("the saved state has no AdamW parameters")
        names = saved.get("names")
        if names is None:
            return saved
        if sorted(names) != sorted(self.adamw_names):
            raise ValueError("the saved AdamW states are those of other parameters")
        at = {n: i for i, n in enumerate(names)}
        lists = {k: v for k, v in saved.items() if isinstance(v, (list, tuple)) and k != "names"}
        for k, v in lists.items():
            if len(v) != len(names):
                raise ValueError(f"one {k} per parameter")
        return {**saved, **{k: [v[at[n]] for n in self.adamw_names] for k, v in lists.items()}}
