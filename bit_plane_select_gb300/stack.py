"""A resident stack of ternary projections: packed planes in HBM plus one
contiguous arena for each of the step's inputs and outputs, so that a batch-1
decode step is one launch (every activation row quantised and every product
computed by the fused kernel; the two-launch path -- quantise, then multiply --
stays available) and an end-to-end step is one host-to-device and one
device-to-host copy around it.

This is the runtime around the kernels for the layer-by-layer decode of
"Tritium: One Weight Format for Ternary Inference ..." -- Why it does not
scale: a token is 210 independent ternary products; here they are issued as
one persistent launch instead of 210 separate dispatches.
"""
from __future__ import annotations

import torch

from . import (MAX_FUSED_K, ActList, ProjList, QProjList, k_pad, payload_bytes,
               trit_gemm_many, trit_pack, trit_quant_act_many, trit_quant_gemv_many)


class TernaryStack:
    def __init__(self, device="cuda"):
        self.device = torch.device(device)
        self.specs = []        # (name, N, K, M, w_scale)
        self.planes = []
        self.finalized = False

    def add(self, w: torch.Tensor, w_scale: float, M: int = 1, name: str = "") -> int:
        """Pack an int8 ternary matrix [N, K] (host or device) and reserve M
        activation rows for it.  Returns its index."""
        assert not self.finalized
        N, K = w.shape
        wd = w.to(self.device, non_blocking=False)
        planes, err = trit_pack(wd, w_scale)
        torch.cuda.current_stream(self.device).synchronize()
        if int(err.item()) != 0:
            raise ValueError(f"projection {name or len(self.specs)}: non-ternary weights")
        del wd
        self.planes.append(planes)
        self.specs.append((name, N, K, M, float(w_scale)))
        return len(self.specs) - 1

    def twin(self) -> "TernaryStack":
        """A finalized stack over the same planes with arenas of its own: two
        twins let consecutive steps use different activation and output
        buffers, so a step's copies can overlap the next step's products."""
        assert self.finalized
        t = TernaryStack.__new__(TernaryStack)
        t.device = self.device
        t.specs = list(self.specs)
        t.planes = self.planes
        t.finalized = False
        t.finalize()
        return t

    def finalize(self):
        """Allocate the arenas and build the launch lists."""
        dev = self.device
        x_el = sum(M * K for _, N, K, M, _ in self.specs)
        q_el = sum(M * k_pad(K) for _, N, K, M, _ in self.specs)
        m_el = sum(M for _, N, K, M, _ in self.specs)
        y_el = sum(M * N for _, N, K, M, _ in self.specs)
        self.x_arena = torch.zeros(x_el, dtype=torch.float32, device=dev)
        self.q_arena = torch.zeros(q_el + 64, dtype=torch.int8, device=dev)
        self.s_arena = torch.zeros(m_el, dtype=torch.float32, device=dev)
        self.y_arena = torch.zeros(y_el, dtype=torch.int32, device=dev)
        self.f_arena = torch.zeros(y_el, dtype=torch.float32, device=dev)
        self.err = torch.zeros(1, dtype=torch.int32, device=dev)
        self.x, self.q, self.s, self.y, self.f = [], [], [], [], []
        xo = qo = so = yo = 0
        for _, N, K, M, _ in self.specs:
            self.x.append(self.x_arena[xo:xo + M * K].view(M, K))
            self.q.append(self.q_arena[qo:qo + M * k_pad(K)].view(M, k_pad(K)))
            self.s.append(self.s_arena[so:so + M])
            self.y.append(self.y_arena[yo:yo + M * N].view(M, N))
            self.f.append(self.f_arena[yo:yo + M * N].view(M, N))
            xo += M * K
            qo += M * k_pad(K)   # multiple of 64 bytes: every row stays 16-byte aligned
            so += M
            yo += M * N
        self.acts = ActList([(self.x[i], self.q[i], self.s[i]) for i in range(len(self.specs))])
        self.projs = ProjList([(self.planes[i], self.specs[i][4], self.q[i], self.s[i],
                                self.specs[i][2], self.y[i], self.f[i])
                               for i in range(len(self.specs))])
        self.fusable = all(M == 1 and K <= MAX_FUSED_K for _, N, K, M, _ in self.specs)
        self.qprojs = None
        if self.fusable:
            self.qprojs = QProjList([(self.planes[i], self.specs[i][4], self.x[i], self.q[i],
                                      self.s[i], self.y[i], self.f[i])
                                     for i in range(len(self.specs))])
        self.finalized = True

    # -- one decode step ------------------------------------------------------

    def quantize(self, stream=None):
        trit_quant_act_many(self.acts, self.err, stream)

    def products(self, stream=None):
        trit_gemm_many(self.projs, self.err, stream)

    def fused(self, stream=None):
        """Quantise and multiply every entry in one launch (M = 1 stacks)."""
        trit_quant_gemv_many(self.qprojs, self.err, stream)

    def step(self, stream=None):
        if self.fusable:
            self.fused(stream)
        else:
            self.quantize(stream)
            self.products(stream)

    def step_two_launch(self, stream=None):
        self.quantize(stream)
        self.products(stream)

    # -- sizes ------------------------------------------------------------------

    @property
    def plane_bytes(self) -> int:
        return sum(payload_bytes(N, K) for _, N, K, M, _ in self.specs)

    @property
    def weights(self) -> int:
        return sum(N * K for _, N, K, M, _ in self.specs)

    def product_bytes(self) -> int:
        """Algorithmic bytes of the product launch: every plane byte read once,
        the int8 activations (K_pad per row) and their scales read, y_i32 and
        y_f32 written."""
        b = 0
        for _, N, K, M, _ in self.specs:
            b += payload_bytes(N, K) + M * k_pad(K) + 4 * M + 8 * M * N
        return b

    def fused_bytes(self) -> int:
        """Algorithmic bytes of the fused launch: planes read once, the fp32
        activations read, int8 codes (K_pad per row) and scales written, y_i32
        and y_f32 written."""
        b = 0
        for _, N, K, M, _ in self.specs:
            b += payload_bytes(N, K) + M * (4 * K + k_pad(K) + 4) + 8 * M * N
        return b

    def quant_bytes(self) -> int:
        """fp32 activations read, int8 codes (K_pad per row) and scales written."""
        return sum(M * (4 * K + k_pad(K) + 4) for _, N, K, M, _ in self.specs)


class LayerChain:
    """The dependency-ordered decode of one token through ternary layers: per
    layer four launches, each reading what the one before wrote --
      1. q, k, v from the layer's input row (quantiser fused),
      2. o from q's fp32 output (the attention output's stand-in: attention
         itself is not a ternary product),
      3. gate and up from o's fp32 output (gate also writes the input scale),
      4. the IntMlp codes of relu(a_gate)^2 a_up and the down product.
    This is the per-matvec ordering of a real token ("Tritium ..." -- Why it
    does not scale): every launch waits for the grid before it (programmatic
    stream serialisation) before it reads its input.  Each layer's input row is
    its own buffer (x[layer]); the residual stream and the norms are not part
    of the ternary path.

    weights: per layer, a dict name -> (int8 [N, K] tensor, w_scale) for the
    seven projections q, k, v, o, gate, up, down.

    mlp_form -- the same bits every way:
      "paired": gate/up as one launch that also publishes max|t| partials
        (trit_mlp_gate_up), then the down product forming the IntMlp codes from
        them while it stages its row (trit_mlp_down): 4 launches per layer;
      "split": gate/up, trit_intmlp_quant, the down product of its int8 codes: 5;
      "fused": gate/up, then every CTA of the down product forms the codes it
        needs, max|t| pass included (trit_intmlp_gemv_many): 4."""

    NAMES = ("q", "k", "v", "o", "gate", "up", "down")
    MLP_FORMS = ("paired", "split", "fused")

    def __init__(self, weights, device="cuda", mlp_form: str = "paired"):
        from . import MlpBlockList, MlpProjList, trit_mlp_tmax_bytes
        if mlp_form not in self.MLP_FORMS:
            raise ValueError(f"mlp_form must be one of {self.MLP_FORMS}")
        self.mlp_form = mlp_form
        self.device = torch.device(device)
        dev = self.device
        self.err = torch.zeros(1, dtype=torch.int32, device=dev)
        self.layers = []
        self.plane_bytes = 0
        for lw in weights:
            P, S, shape = {}, {}, {}
            for name in self.NAMES:
                w, ws = lw[name]
                planes, err = trit_pack(w.to(dev), ws)
                if int(err.item()) != 0:
                    raise ValueError(f"{name}: non-ternary weights")
                P[name], S[name], shape[name] = planes, float(ws), tuple(w.shape)
                self.plane_bytes += planes.numel()
            Nq, K = shape["q"]
            Nk, Nv = shape["k"][0], shape["v"][0]
            No, Ko = shape["o"]
            Nf, Kg = shape["gate"]
            Nd, Kd = shape["down"]
            if Ko != Nq or Kg != No or Kd != Nf or shape["up"] != shape["gate"]:
                raise ValueError("layer shapes do not chain")
            L = {"P": P, "S": S}
            L["x"] = torch.zeros(K, dtype=torch.float32, device=dev)
            for name, n in (("q", Nq), ("k", Nk), ("v", Nv), ("o", No), ("down", Nd)):
                L["y_" + name] = torch.zeros(n, dtype=torch.int32, device=dev)
                L["f_" + name] = torch.zeros(n, dtype=torch.float32, device=dev)
            L["a_gate"] = torch.zeros(Nf, dtype=torch.int32, device=dev)
            L["a_up"] = torch.zeros(Nf, dtype=torch.int32, device=dev)
            L["s_gu"] = torch.zeros(1, dtype=torch.float32, device=dev)
            # the planes are packed (and the stream synchronised) here, before any
            # launch of the chain: every list may read them ahead of its grid dependency
            L["qkv"] = QProjList([(P[n], S[n], L["x"], None, None, L["y_" + n], L["f_" + n])
                                  for n in ("q", "k", "v")], planes_ready=True)
            L["o"] = QProjList([(P["o"], S["o"], L["f_q"], None, None, L["y_o"], L["f_o"])],
                               planes_ready=True)
            L["gu"] = QProjList([(P["gate"], S["gate"], L["f_o"], None, L["s_gu"], L["a_gate"], None),
                                 (P["up"], S["up"], L["f_o"], None, None, L["a_up"], None)],
                                planes_ready=True)
            L["down"] = MlpProjList([(P["down"], S["down"], L["a_gate"], L["a_up"], L["s_gu"],
                                      S["gate"], S["up"], None, None, L["y_down"], L["f_down"])])
            L["h"] = torch.zeros(k_pad(Kd), dtype=torch.int8, device=dev)
            L["s_h"] = torch.zeros(1, dtype=torch.float32, device=dev)
            L["down_i8"] = ProjList([(P["down"], S["down"], L["h"], L["s_h"], Kd, L["y_down"],
                                      L["f_down"])], planes_ready=True)
            L["tmax"] = torch.zeros(trit_mlp_tmax_bytes(Nf), dtype=torch.uint8, device=dev)
            L["mlp"] = MlpBlockList([(P["gate"], P["up"], P["down"], S["gate"], S["up"], S["down"],
                                      L["f_o"], L["s_gu"], L["a_gate"], L["a_up"], L["tmax"], None,
                                      None, L["y_down"], L["f_down"])], planes_ready=True)
            self.layers.append(L)

    @property
    def x(self):
        return [L["x"] for L in self.layers]

    def step(self, stream=None):
        """One token through every layer: 4 launches per layer (5 for "split")."""
        from . import trit_intmlp_gemv_many, trit_intmlp_quant, trit_mlp_down, trit_mlp_gate_up
        for L in self.layers:
            trit_quant_gemv_many(L["qkv"], self.err, stream)
            trit_quant_gemv_many(L["o"], self.err, stream)
            if self.mlp_form == "paired":
                trit_mlp_gate_up(L["mlp"], self.err, stream)
                trit_mlp_down(L["mlp"], self.err, stream)
                continue
            trit_quant_gemv_many(L["gu"], self.err, stream)
            if self.mlp_form == "fused":
                trit_intmlp_gemv_many(L["down"], self.err, stream)
            else:
                S = L["S"]
                trit_intmlp_quant(L["a_gate"][None, :], L["a_up"][None, :], S["gate"], S["up"],
                                  L["s_gu"], L["h"][None, :], L["s_h"], stream)
                trit_gemm_many(L["down_i8"], self.err, stream)

    @property
    def stages_per_step(self) -> int:
        return 4 * len(self.layers)

    @property
    def launches_per_step(self) -> int:
        return (5 if self.mlp_form == "split" else 4) * len(self.layers)

    def step_bytes(self) -> int:
        """Algorithmic bytes of one token: every plane byte read once; per
        launch its fp32 (or int32) inputs read and int32 + fp32 outputs written."""
        b = self.plane_bytes
        for L in self.layers:
            K = L["x"].numel()
            nq, nk, nv = (L["y_" + n].numel() for n in ("q", "k", "v"))
            no, nf, nd = L["y_o"].numel(), L["a_gate"].numel(), L["y_down"].numel()
            b += 4 * K + 8 * (nq + nk + nv)          # qkv: x read, y + f written
            b += 4 * nq + 8 * no                     # o: q's f read
            b += 4 * no + 4 + 8 * nf                 # gate/up: o's f read, scale, a_gate + a_up
            b += 8 * nf + 4 + 8 * nd                 # down: a_gate + a_up read, scale
        return b


class ServedStack:
    """Ternary layers with attention between their products, for a batch of
    sequences that decode (or verify drafts) behind a shared prefix.  Per layer:
      1. norm folded into the quantiser, q, k and v products,
      2. trit_kv_append: rotation, optional head norms, the cache append,
      3. trit_attn_paged (fp32 out), quantised, the o product, residual;
      4. norm folded into the quantiser, gate and up, trit_intmlp_quant, the down
         product, residual.
    Each layer owns a paged cache; a plan (see `plan`) holds the buffers and
    prepared lists of one KvBatch, so the prefix's prompt and the decode steps
    are two plans over the same caches.

    With cache_bits=4 the caches hold 4 bits (Kv4Cache) and 2. and 3. are
    trit_kv4_append and trit_attn_paged4; whole prompts of different lengths then go in
    as packed rows (see `prompt_plan`): trit_kv4_append, trit_kv4_read and trit_attn_prompt,
    so that prompts and single tokens attend to the same cached values.

    weights: per layer, name -> (int8 [N, K] tensor, w_scale) for q, k, v, o, gate,
    up, down, plus "attn_gain" and "mlp_gain" (fp32 [K] norm gains).  rope: a
    Rope; pages and page_size: of every layer's cache; dtype: of the queries and of
    16-bit keys and values."""

    NAMES = LayerChain.NAMES

    def __init__(self, weights, head_dim: int, rope, pages: int, page_size: int,
                 dtype=torch.bfloat16, eps: float = 1e-5, device="cuda", cache_bits: int = 16):
        from . import Kv4Cache, KvCache
        if cache_bits not in (4, 16):
            raise ValueError("cache_bits must be 4 or 16")
        self.cache_bits, self.dtype = cache_bits, dtype
        self.device, self.head_dim, self.rope, self.eps = torch.device(device), head_dim, rope, float(eps)
        self.layers = []
        sizes = self._sizes(weights, head_dim)
        for lw, (K, F, heads) in zip(weights, sizes):
            P, S = {}, {}
            for name in self.NAMES:
                w, ws = lw[name]
                planes, err = trit_pack(w.to(self.device), ws)
                if int(err.item()) != 0:
                    raise ValueError(f"{name}: non-ternary weights")
                P[name], S[name] = planes, float(ws)
            if cache_bits == 4:
                cache = Kv4Cache.empty(pages, heads["k"], page_size, head_dim, self.device)
            else:
                cache = KvCache(*(torch.zeros((pages, heads["k"], page_size, head_dim), dtype=dtype, device=self.device)
                                  for _ in range(2)))
            gains = [lw[g].to(device=self.device, dtype=torch.float32) for g in ("attn_gain", "mlp_gain")]
            self.layers.append({"P": P, "S": S, "K": K, "F": F, "heads": heads, "cache": cache,
                                "attn_gain": gains[0], "mlp_gain": gains[1]})
        self.err = torch.zeros(1, dtype=torch.int32, device=self.device)

    @classmethod
    def _sizes(cls, weights, head_dim: int):
        """(K, F, heads) of every layer: each fits itself, and all take rows of one width."""
        sizes = []
        for lw in weights:
            shape = {name: tuple(lw[name][0].shape) for name in cls.NAMES}
            K, F = shape["q"][1], shape["gate"][0]
            heads = {n: shape[n][0] // head_dim for n in ("q", "k", "v")}
            if (shape["o"] != (K, shape["q"][0]) or shape["k"] != shape["v"] or shape["gate"] != (F, K) or
                    shape["up"] != (F, K) or shape["down"] != (K, F) or shape["k"][1] != K or
                    any(heads[n] * head_dim != shape[n][0] for n in heads) or (sizes and K != sizes[0][0])):
                raise ValueError("layer shapes do not chain")
            if any(lw[g].numel() != K for g in ("attn_gain", "mlp_gain")):
                raise ValueError(f"a layer's gains must hold {K} values")
            sizes.append((K, F, heads))
        if not sizes:
            raise ValueError("a stack needs a layer")
        return sizes

    def plan(self, batch):
        """Buffers and prepared calls for the T new tokens of every sequence of `batch`."""
        from . import Append4Job, AppendJob, Attn4Job, AttnJob, trit_attn_paged, trit_attn_paged4, trit_kv4_append, trit_kv_append
        four = self.cache_bits == 4
        plan, workspaces = [], {}
        for L in self.layers:
            hq, hk, D = L["heads"]["q"], L["heads"]["k"], self.head_dim
            B = self._buffers(L, batch.B * batch.T, (batch.B, batch.T, hq, D))
            B["append"] = (Append4Job if four else AppendJob)(L["cache"], batch, self.rope, B["q"], B["k"], B["v"], B["q_rot"])
            # (layers of one size take turns with a workspace, which may hold a whole prefix)
            B["attend"] = (Attn4Job if four else AttnJob)(L["cache"], batch, B["q_rot"], B["attn"], workspace=workspaces.get((hq, hk)))
            workspaces[hq, hk] = B["attend"].workspace
            B["calls"] = [(trit_kv4_append if four else trit_kv_append, B["append"]),
                          (trit_attn_paged4 if four else trit_attn_paged, B["attend"])]
            plan.append(B)
        return plan

    def prompt_plan(self, batch, rows: int, starts, keys: int, key_starts):
        """Buffers and prepared calls for whole prompts as packed rows (4-bit caches): of x's
        `rows` rows, sequence b's new tokens are starts[b] .. starts[b+1] - 1 (starts [B + 1]
        int32; at most batch.T each), and its prefix_len + lens[b] keys, the new ones
        last, take key_starts[b] .. key_starts[b+1] - 1 of `keys` (key_starts
        [B + 1] int32).  Both are read when a step runs, as the batch's tables are."""
        from . import Append4Job, PromptJob, Read4Job, trit_attn_prompt, trit_kv4_append, trit_kv4_read
        if self.cache_bits != 4:
            raise ValueError("packed prompts need caches of 4 bits")
        plan, packed, shared = [], {}, {}
        for L in self.layers:
            hq, hk, D = L["heads"]["q"], L["heads"]["k"], self.head_dim
            B = self._buffers(L, rows, (rows, hq, D), shared)
            for name in ("q_rot", "attn"):          # rows of no sequence start as 0
                B[name].zero_()
            if hk not in packed:                    # the layers take turns
                packed[hk] = [torch.zeros((keys, hk, D), dtype=self.dtype, device=self.device) for _ in range(2)]
            k, v = packed[hk]
            B["append"] = Append4Job(L["cache"], batch, self.rope, B["q"], B["k"], B["v"], B["q_rot"], starts=starts)
            B["read"] = Read4Job(L["cache"], batch, k, v, key_starts)
            B["attend"] = PromptJob(B["q_rot"], k, v, B["attn"], starts, key_starts)
            B["calls"] = [(trit_kv4_append, B["append"]), (trit_kv4_read, B["read"]), (trit_attn_prompt, B["attend"])]
            plan.append(B)
        return plan

    def _buffers(self, L, M: int, q_shape, shared=None):
        """A layer's buffers and products for M rows.  With `shared`, what no later layer reads is taken
        from there, where another of the same size has left it."""
        D, dev = self.head_dim, self.device

        def buf(*shape, dtype=torch.float32):
            return torch.empty(shape, dtype=dtype, device=dev)
        K, F, hq, hk, P, S = L["K"], L["F"], L["heads"]["q"], L["heads"]["k"], L["P"], L["S"]
        i8, i32, f32 = torch.int8, torch.int32, torch.float32
        B = {"q_rot": buf(*q_shape, dtype=self.dtype), "attn": buf(*q_shape)}
        for name, width, dtype in (("x_i8", k_pad(K), i8), ("a_i8", k_pad(hq * D), i8), ("h_i8", k_pad(F), i8), ("s", 0, f32),
                                   ("sa", 0, f32), ("sh", 0, f32), ("q", hq * D, f32), ("k", hk * D, f32), ("v", hk * D, f32),
                                   ("o", K, f32), ("down", K, f32), ("gate", F, i32), ("up", F, i32)):
            at = (name, width)
            if shared is None or at not in shared:
                B[name] = buf(*((M, width) if width else (M,)), dtype=dtype)
                if shared is not None:
                    shared[at] = B[name]
            else:
                B[name] = shared[at]
        B["qkv_list"] = ProjList([(P[n], S[n], B["x_i8"], B["s"], K, None, B[n]) for n in "qkv"])
        B["o_list"] = ProjList([(P["o"], S["o"], B["a_i8"], B["sa"], hq * D, None, B["o"])])
        B["gu_list"] = ProjList([(P[n], S[n], B["x_i8"], B["s"], K, B[n], None) for n in ("gate", "up")])
        B["down_list"] = ProjList([(P["down"], S["down"], B["h_i8"], B["sh"], F, None, B["down"])])
        return B

    def step(self, plan, x, stream=None):
        """x [rows, K] fp32, the new tokens' rows (B*T of them, or a prompt plan's), through every
        layer in place."""
        from . import trit_intmlp_quant, trit_quant_act, trit_quant_act_folded
        if len(plan) != len(self.layers) or tuple(x.shape) != tuple(plan[0]["o"].shape):
            raise ValueError("x must be [B*T, K] of the plan's batch")
        with torch.cuda.stream(stream) if stream is not None else torch.cuda.stream(torch.cuda.current_stream()):
            for L, B in zip(self.layers, plan):
                trit_quant_act_folded(x, L["attn_gain"], self.eps, B["x_i8"], B["s"], self.err)
                trit_gemm_many(B["qkv_list"], self.err)
                for call, job in B["calls"]:
                    call(job, self.err)
                trit_quant_act(B["attn"].view(x.shape[0], -1), B["a_i8"], B["sa"], self.err)
                trit_gemm_many(B["o_list"], self.err)
                x += B["o"]
                trit_quant_act_folded(x, L["mlp_gain"], self.eps, B["x_i8"], B["s"], self.err)
                trit_gemm_many(B["gu_list"], self.err)
                trit_intmlp_quant(B["gate"], B["up"], L["S"]["gate"], L["S"]["up"], B["s"], B["h_i8"], B["sh"])
                trit_gemm_many(B["down_list"], self.err)
                x += B["down"]
        return x
