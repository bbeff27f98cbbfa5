"""A decode step as a server runs it: the synthetic Qwen3-shaped step with its
KV cache, attention and logit rules.

    plan   page for each request's new token          nvfp4_kv_plan
    per layer, between the qkv and o projections:
        K, V columns of qkv -> the 4-bit cache        nvfp4_kv_append
        q columns over it -> BF16                     nvfp4_kv_attention
        -> NVFP4                                      nvfp4_quantize_act
    logits -> penalties, biases, grammar masks        nvfp4_process_logits (in place)
    -> ReSET sampler of the rows with a request; the token joins its request's history

Every layer has a cache of its own; one page table serves them all (a page has
the same number in each).  Requests come with `start` (prompts, whose K and V
rows the caller gives) and go with `end`, whose pages the next requests get.
No rotary positions: the step is synthetic, and `plan.positions` (of the rows
that get a token, one behind the other) is where a model takes them from.  The step itself (`run`, `capture`) reads lengths, tables
and histories on the device only, so one captured graph follows any requests.
"""
import torch

from . import api
from .decode_step import DecodeStep


class ServingStep(DecodeStep):
    def __init__(self, M: int, layers: int, heads: int, kv_heads: int, head_dim: int = 128, page_size: int = 64,
                 num_pages: int = 1024, max_len: int = 32768, k_global: float = 1.0, v_global: float = 1.0, **kw):
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
        # views and buffers of the attention
        cut = heads * head_dim
        self.q = self.y_qkv[:, :cut].unflatten(-1, (heads, head_dim))
        self.k = self.y_qkv[:, cut:cut + kv_heads * head_dim].unflatten(-1, (kv_heads, head_dim))
        self.v = self.y_qkv[:, cut + kv_heads * head_dim:].unflatten(-1, (kv_heads, head_dim))
        self.attn = torch.empty((M, heads, head_dim), dtype=torch.bfloat16, device=dev)
        need = api.nvfp4_kv_attention_workspace_bytes(M, M, heads, kv_heads, head_dim)
        self.attn_ws = torch.zeros(need, dtype=torch.uint8, device=dev)

    # ---- requests -----------------------------------------------------------------
    def start(self, prompts: dict, keys, values):
        """New requests: {row: prompt tokens (1-D int32 on the device)}; keys[layer], values[layer]: their K and V
        rows [total, kv_heads, head_dim], packed in row order.  Returns the plan (its info: refused, tokens): a prompt
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
            api.nvfp4_kv_append(k, v, plan.slots, cache)
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
        api.nvfp4_kv_append(self.k, self.v, self.slots, cache, stream=stream)
        api.nvfp4_kv_attention(self.q, cache, self.table, self.attn_lens, out=self.attn, workspace=self.attn_ws,
                               stream=stream)
        api.nvfp4_quantize_act(self.attn.view(self.M, self.k_o), out=self.xq_o, stream=stream)

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
