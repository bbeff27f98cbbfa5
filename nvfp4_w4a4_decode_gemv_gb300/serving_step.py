"""A decode step as a server runs it: the synthetic Qwen3-shaped step with its
KV cache, attention and logit rules.

    plan   page for each request's new token          nvfp4_kv_plan
    per layer, between the qkv and o projections:
        K, V columns of qkv -> the 4-bit cache        nvfp4_kv_append, or with positions, q and K rotated by them,
                                                      nvfp4_kv_append_rope
        q columns over it -> BF16                     nvfp4_kv_attention
        -> NVFP4                                      nvfp4_quantize_act
    per layer, with experts, instead of its gate_up and down projections:
        router logits of the normalized rows          nvfp4_bf16_gemv_tc
        -> the chosen experts and the pairs' plan     nvfp4_moe_route
        gate and up of each, SiLU(gate) up            nvfp4_moe_gate_up
        -> NVFP4                                      nvfp4_quantize_act
        down, summed with the weights                 nvfp4_moe_down
    logits -> penalties, biases, grammar masks        nvfp4_process_logits (in place)
    -> ReSET sampler of the rows with a request; the token joins its request's history

Every layer has a cache of its own; one page table serves them all (a page has
the same number in each).  Requests come with `start` (prompts, whose K and V
rows the caller gives) and go with `end`, whose pages the next requests get.
Positions are optional, as the step is synthetic (`rotary`); a token's position is its
place in its request.  The step itself (`run`, `capture`) reads lengths, tables
and histories on the device only, so one captured graph follows any requests.
"""
import torch

from . import api
from .decode_step import DecodeStep


class ServingStep(DecodeStep):
    """rotary: the base of the rotation's angles (None: no positions), of the first `rotated` elements of a head (all by
    default), in pairs of `rope_style`.  experts: their number (0: dense layers); `shapes` then holds the gate_up and down
    projections of one expert, and `router` what nvfp4_moe_route takes (top_k, score, groups, ...); `route_bias[layer]` may
    be set to a float32 [experts] tensor."""

    def __init__(self, M: int, layers: int, heads: int, kv_heads: int, head_dim: int = 128, page_size: int = 64,
                 num_pages: int = 1024, max_len: int = 32768, k_global: float = 1.0, v_global: float = 1.0,
                 rotary: float | None = None, rotated: int | None = None, rope_style: str = "halves", experts: int = 0,
                 router: dict | None = None, **kw):
        self.experts, self.router, self.routers = experts, dict(router or {"top_k": 1}), []
        super().__init__(M, layers, **kw)
        if self.k_o != heads * head_dim or self.n_qkv != (heads + 2 * kv_heads) * head_dim:
            raise ValueError("the qkv and o shapes do not fit the heads")
        dev, i32 = self.device, dict(dtype=torch.int32, device=self.device)
        self.heads, self.kv_heads, self.head_dim, self.page_size, self.max_len = heads, kv_heads, head_dim, page_size, max_len
        self.caches = [api.NVFP4KVCache.empty(num_pages, page_size, kv_heads, head_dim, k_global, v_global, dev)
                       for _ in range(layers)]
        # requests: keys held, page table, stack of free pages
        self.lens = torch.zeros(M, **i32)
        self.active = torch.zeros(M, **i32)              # 1: the row has a request
        self.wanted = torch.zeros(M, **i32)              # 1: and its history has room for a token
        self.slots = torch.full((M,), -1, **i32)         # of each row's new token, -1: none, or no page for it
        self.live = torch.zeros(M, dtype=torch.bool, device=dev)   # rows with a slot: the step is theirs
        self.attn_lens = torch.zeros(M, **i32)           # keys that a live row sees, 0 for the others
        self.h_live = torch.zeros_like(self.h_in)        # h_in of the live rows, 0 for the others
        self.none, self.zero = torch.zeros((), **i32), torch.zeros((), device=dev)
        self.table = torch.full((M, -(-max_len // page_size)), -1, **i32)
        self.free_pages = torch.arange(num_pages, **i32)
        self.free_count = torch.full((1,), num_pages, **i32)
        self.plan = api.KVPlan.empty(M, M, dev, free_count=self.free_count)
        # token histories and rules
        self.tokens = torch.zeros((M, max_len), **i32)
        self.n_tokens, self.n_prompt = torch.zeros(M, **i32), torch.zeros(M, **i32)
        self.rows = torch.arange(M, device=dev)
        f32 = dict(dtype=torch.float32, device=dev)
        self.repetition, self.presence, self.frequency = torch.ones(M, **f32), torch.zeros(M, **f32), torch.zeros(M, **f32)
        self.bias_ids = self.bias_values = self.mask = self.mask_rows = None
        self.rope, self.rope_style = None, rope_style
        if rotary is not None:
            self.rope = api.rope_table(max_len, rotated or head_dim, rotary, device=dev)
            self.q_turned = torch.empty((M, heads, head_dim), dtype=torch.bfloat16, device=dev)
        if experts:
            shared = kw.get("share_weights")
            g = torch.Generator(device=dev)
            g.manual_seed(kw.get("seed", 0) * 100003 + 99989)
            self.routers = shared.routers if shared is not None else [
                (torch.randn((experts, self.hidden), generator=g, device=dev) / self.hidden ** 0.5).to(torch.bfloat16)
                for _ in range(layers)]
            self.route_bias = [None] * layers
            top_k = self.router["top_k"]
            self.route_logits = torch.empty((M, experts), **f32)
            self.routing = api.MoERouting.empty(M, top_k, experts, dev)
            self.h_mid = torch.empty((M * top_k, self.k_d), dtype=torch.bfloat16, device=dev)
            self.xq_d = api.NVFP4Tensor.empty(M * top_k, self.k_d, dev)
            need = api.nvfp4_bf16_gemv_workspace_bytes(M, experts, self.hidden)
            if self.ws.numel() < need:
                self.ws = torch.zeros(need, dtype=torch.uint8, device=dev)
        # views and buffers of the attention
        cut = heads * head_dim
        self.q = self.y_qkv[:, :cut].unflatten(-1, (heads, head_dim))
        self.k = self.y_qkv[:, cut:cut + kv_heads * head_dim].unflatten(-1, (kv_heads, head_dim))
        self.v = self.y_qkv[:, cut + kv_heads * head_dim:].unflatten(-1, (kv_heads, head_dim))
        self.attn = torch.empty((M, heads, head_dim), dtype=torch.bfloat16, device=dev)
        need = api.nvfp4_kv_attention_workspace_bytes(M, M, heads, kv_heads, head_dim)
        self.attn_ws = torch.zeros(need, dtype=torch.uint8, device=dev)

    def _make_weight(self, name, K, N, g):
        if not self.experts or name not in ("gate_up", "down"):
            return super()._make_weight(name, K, N, g)
        rows = [self._random_weight(K, N, g) for _ in range(self.experts)]
        stack = [torch.stack([getattr(w, part) for w in rows]) for part in ("codes", "scales", "global_scale")]
        return api.nvfp4_moe_pack_weights(stack[0], stack[1], stack[2].view(-1), gated=name == "gate_up"), rows

    # ---- requests -----------------------------------------------------------------
    def start(self, prompts: dict, keys, values):
        """New requests: {row: prompt tokens (1-D int32 on the device)}; keys[layer], values[layer]: their K and V
        rows [total, kv_heads, head_dim], packed in row order (K not yet rotated: positions turn it here).  Returns the plan (its info: refused, tokens): a prompt
        without room has kv_lens[row] = 0 there, and its row stays without a request."""
        new = torch.zeros(self.M, dtype=torch.int32)
        for row, ids in prompts.items():
            if not 0 <= row < self.M:
                raise ValueError(f"there is no row {row}")
            if ids.numel() > self.max_len:
                raise ValueError(f"the prompt of row {row} is longer than max_len")
            new[row] = ids.numel()
        held = self.active.tolist()
        for row in prompts:
            if held[row]:
                raise ValueError(f"row {row} has a request")
        plan = api.KVPlan.empty(self.M, int(new.sum()), self.device, free_count=self.free_count)
        new = new.to(self.device)
        api.nvfp4_kv_plan(self.lens, new, self.table, self.free_pages, self.free_count, self.page_size, out=plan)
        given = torch.tensor([row in prompts for row in range(self.M)], device=self.device)
        taken = given & (plan.kv_lens == self.lens + new)
        for cache, k, v in zip(self.caches, keys, values):
            if self.rope is None:
                api.nvfp4_kv_append(k, v, plan.slots, cache)
            else:
                api.nvfp4_kv_append_rope(None, k, v, plan.positions, plan.slots, cache, self.rope, self.rope_style)
        self.lens.copy_(plan.kv_lens)
        self.sampler.restart(taken)
        for row, ids in prompts.items():
            self.tokens[row, :ids.numel()] = ids         # (of no meaning while n_tokens is 0)
        for t, value in ((self.n_tokens, new), (self.n_prompt, new), (self.active, 1)):
            t.copy_(torch.where(taken, value, t))
        return plan

    def end(self, ended: torch.Tensor):
        """Requests with ended[row] != 0 (uint8 [M]) leave; their pages are free again."""
        api.nvfp4_kv_release(self.lens, ended, self.table, self.free_pages, self.free_count, self.page_size)
        stay = (ended == 0).to(torch.int32)
        for t in (self.lens, self.n_tokens, self.n_prompt, self.active):
            t.mul_(stay)

    # ---- the step -----------------------------------------------------------------
    def _input(self):
        return self.h_live

    def _attend(self, layer: int, stream):
        cache = self.caches[layer]
        q = self.q
        if self.rope is None:
            api.nvfp4_kv_append(self.k, self.v, self.slots, cache, stream=stream)
        else:                                            # a live row's new token stands behind the keys it holds
            q = api.nvfp4_kv_append_rope(q, self.k, self.v, self.lens, self.slots, cache, self.rope, self.rope_style,
                                         q_out=self.q_turned, stream=stream)
        api.nvfp4_kv_attention(q, cache, self.table, self.attn_lens, out=self.attn, workspace=self.attn_ws,
                               stream=stream)
        api.nvfp4_quantize_act(self.attn.view(self.M, self.k_o), out=self.xq_o, stream=stream)

    def _mlp(self, layer: int, stream, trace):
        if not self.experts:
            return super()._mlp(layer, stream, trace)
        w = self.weights[layer]
        api.nvfp4_rms_norm_quantize(self.y_o, eps=self.eps, out=self.xq_gu, r_out=self.r, stream=stream)
        api.nvfp4_bf16_gemv_tc(self.r, self.routers[layer], y=self.route_logits, workspace=self.ws, stream=stream)
        api.nvfp4_moe_route(self.route_logits, bias=self.route_bias[layer], rows=self.live, out=self.routing, stream=stream,
                            **self.router)
        api.nvfp4_moe_gate_up(self.xq_gu, w["gate_up"], self.routing, out=self.h_mid, stream=stream)
        if trace is not None:
            trace[-1]["h_mid"] = self.h_mid.clone()
        api.nvfp4_quantize_act(self.h_mid, out=self.xq_d, stream=stream)
        api.nvfp4_moe_down(self.xq_d, w["down"], self.routing, y=self.h, stream=stream)

    def _sample(self, stream):
        api.nvfp4_process_logits(self.logits, self.tokens, self.n_tokens, self.n_prompt, self.repetition, self.presence,
                                 self.frequency, self.bias_ids, self.bias_values, self.mask, self.mask_rows,
                                 out=self.logits, stream=stream)
        return self.sampler(self.logits, self.step_start, self.u, stream=stream, rows=self.live)

    def run(self, stream=None, trace=None):
        """One decode step of every request: h_in, u, step_start -> sampler.token; lengths and histories move on, but
        not those of a request for whose token there is no page, or whose history is full (max_len tokens).  Such rows,
        and those without a request, are zero throughout: they change no result of the others (whose activations they
        share a scale with), no state and no output.  A row whose rules leave no token gets -1, which its history
        holds but does not count (device error bit 4)."""
        with torch.cuda.stream(stream):
            # a row with a request and room in its history gets a token
            torch.mul(self.active, self.n_tokens < self.max_len, out=self.wanted)
            api.nvfp4_kv_plan(self.lens, self.wanted, self.table, self.free_pages, self.free_count, self.page_size,
                              out=self.plan, stream=stream)
            # the plan's tokens are those of the wanted rows, one behind the other
            packed = self.plan.slots[self.plan.cu_q[:-1].clamp(max=self.M - 1).long()]
            self.slots.copy_(torch.where(self.wanted > 0, packed, -1))
            torch.ge(self.slots, 0, out=self.live)
            torch.where(self.live, self.plan.kv_lens, self.none, out=self.attn_lens)
            torch.where(self.live[:, None], self.h_in, self.zero, out=self.h_live)
            out = super().run(stream, trace)
            self.lens.copy_(self.plan.kv_lens)
            at = self.n_tokens.clamp(max=self.max_len - 1).long()
            self.tokens[self.rows, at] = torch.where(self.live, self.sampler.token, self.tokens[self.rows, at])
            self.n_tokens.add_(self.live.to(torch.int32))
        return out
