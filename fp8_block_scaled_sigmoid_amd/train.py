"""One MoE block trained in bf16: norm, router, routed and shared SwiGLU experts,
combine, norm, gate and residual sum, forwards and backwards.

The heavy steps are the library's entry points; PyTorch does the small gather
and scatter work on [T, k] gates.  Weights are bf16 (the norms' and the gate's
float32), gradients float32 in buffers that stay where they are, so that one
``GradList`` over them serves every step:

    block = MoEBlock(weights, k=8)
    r, _, saved = block.forward(x)
    dx, _ = block.backward(saved, dr)              # fills block.grads
    norm, coef = block.clip(1.0)

In a chain of blocks the boundary between two of them is one pass each way: the
first one forms the second one's norm, and takes back that norm's gradient.

    r1, h1, s1 = one.forward(x, next_w_pre=two.w.w_pre)
    r2, _, s2 = two.forward(r1, h=h1)
    dr1, _, dh1 = two.backward(s2, dr2, through_norm=False)
    dx, _ = one.backward(s1, dr1, dh_next=dh1, next_w_pre=two.w.w_pre,
                         dw_next=two.grads["w_pre"])

With balance_alpha the router's balance loss of each sequence is formed in the
forward pass and its gradient joins that of the gates in the backward pass:

    block = MoEBlock(weights, k=8, balance_alpha=1e-4)
    r, _, saved = block.forward(x, seq_offsets=offsets)
    loss = task_loss + block.balance_loss(saved).sum()
"""
import torch

from . import (GradList, moe_balance_loss, moe_block_norm, moe_block_norm_backward, moe_combine,
               moe_grad_clip, moe_grouped_gemm_bf16, moe_grouped_wgrad_bf16, moe_permute,
               moe_route_topk, moe_router_backward, moe_swiglu, moe_swiglu_backward)


class BlockWeights:
    """Device weights of a block: w_router bf16 [N,H], bias float32 [N] (routing
    only, not trained by gradients), w1 bf16 [N+1,2I,H] (gate rows, then up
    rows), w2 bf16 [N+1,H,I] (expert N is the shared one), w_pre and w_post
    float32 [H] (the norms before and after the experts), gate float32 [H]."""

    trained = ("w_router", "w1", "w2", "w_pre", "w_post", "gate")

    def __init__(self, w_router, bias, w1, w2, w_pre, w_post, gate):
        self.w_router, self.bias, self.w1, self.w2 = w_router, bias, w1, w2
        self.w_pre, self.w_post, self.gate = w_pre, w_post, gate
        self.N, self.H = w_router.shape
        self.I = w2.shape[2]
        if tuple(w1.shape) != (self.N + 1, 2 * self.I, self.H) or \
                tuple(w2.shape) != (self.N + 1, self.H, self.I):
            raise ValueError("w1 and w2: need [N+1, 2I, H] and [N+1, H, I]")


def router_gradient(dgate, gates, s):
    """Gradient of the picked logits z from that of the gates g = s / sum s over
    a token's picks, s = sigmoid(z): dz_i = g_i (1 - s_i) (dg_i - sum_j dg_j g_j),
    without a division, so that tiny scores lose nothing.  Where all scores are
    zero the router gives 1/k whatever z is, and dz is zero.  All float32 [T,k]."""
    dz = gates * (1.0 - s) * (dgate - (dgate * gates).sum(1, keepdim=True))
    return torch.where(s.sum(1, keepdim=True) > 0.0, dz, torch.zeros_like(dz))


class MoEBlock:
    """r = alpha x + beta gate rmsnorm(experts(rmsnorm(x, w_pre)), w_post).
    balance_alpha: the weight of the router's balance loss (0: there is none)."""

    def __init__(self, weights, k, alpha=1.0, beta=1.0, eps=1e-6, balance_alpha=0.0):
        self.w, self.k, self.alpha, self.beta, self.eps = weights, k, alpha, beta, eps
        self.balance_alpha = balance_alpha
        dev = weights.w1.device
        self.grads = {n: torch.zeros(getattr(weights, n).shape, dtype=torch.float32, device=dev)
                      for n in weights.trained}
        # every expert's gradient is a tensor of its own, as an optimizer holds them
        self.list = GradList([t for n in weights.trained
                              for t in (self.grads[n] if self.grads[n].dim() == 3
                                        else [self.grads[n]])])

    def forward(self, x, h=None, next_w_pre=None, seq_offsets=None, token_mask=None):
        """x [T,H] the residual stream (bf16 or float32).  h: x already normalised
        with w_pre by the block before (its next_w_pre), else None.  Returns
        (r, h_next or None, saved): with next_w_pre the next block's norm is
        formed in the same pass as r.  seq_offsets int32 [S+1] and token_mask [T] (on
        the device; None: one sequence, all tokens) are the balance loss's, and are not
        read where balance_alpha is 0: without that loss nothing depends on them."""
        w, T = self.w, x.shape[0]
        if h is None:
            h = torch.empty(T, w.H, dtype=torch.bfloat16, device=x.device)
            moe_block_norm(x, w_pre=w.w_pre, eps=self.eps, h=h)
        idx, gates, scores = moe_route_topk(h, w.w_router, w.bias, self.k)
        counts, offsets, row_of, token_of = moe_permute(idx, w.N, True)
        offsets = offsets[:w.N + 2]
        R = token_of.numel()
        a = moe_grouped_gemm_bf16(h, w.w1, offsets, R, a_row_index=token_of)
        rows = moe_grouped_gemm_bf16(moe_swiglu(a), w.w2, offsets, R)
        b = moe_combine(rows, gates, row_of, T * self.k)
        r, h_next = moe_block_norm(x, b, w_pre=next_w_pre, w_post=w.w_post, gate=w.gate,
                                   alpha=self.alpha, beta=self.beta, eps=self.eps)
        saved = (x, h, idx, gates, scores, offsets, row_of, token_of, a, b, r)
        if self.balance_alpha:
            loss, stats = moe_balance_loss(scores, idx, seq_offsets, token_mask, self.balance_alpha)
            saved += ((loss, stats, seq_offsets, token_mask, self.balance_alpha),)
        return r, h_next, saved + (counts,)

    def balance_loss(self, saved):
        """The balance loss of each sequence of a forward pass, float32 [S]."""
        if len(saved) != 13:
            raise ValueError("the forward pass had no balance loss: balance_alpha was 0")
        return saved[11][0]

    def backward(self, saved, dr, dh_next=None, next_w_pre=None, dw_next=None, through_norm=True,
                 dbalance=None):
        """dr: the gradient of r; dh_next: of h_next, when the forward pass formed
        it and the next block went back with through_norm=False (otherwise dr
        holds that part already).  Overwrites self.grads and returns (dx,
        dw_next): the gradient of x, and of next_w_pre (None without dh_next;
        written to dw_next where that is given).  With through_norm=False, for a
        block whose h was given, returns (dx, dw_next, dh): the gradients of x
        and h apart, and self.grads["w_pre"] is left to the block before.  dbalance:
        float32 [S], the gradient of the balance losses (None: 1 each), whose weight
        is the forward pass's balance_alpha."""
        w, g = self.w, self.grads
        balance = saved[11] if len(saved) == 13 else None
        if balance is None and dbalance is not None:
            raise ValueError("dbalance belongs to a forward pass with a balance loss")
        x, h, idx, gates, scores, offsets, row_of, token_of, a, b, r = saved[:11]
        T, R = x.shape[0], token_of.numel()
        dx, db, dw_next, _, _ = moe_block_norm_backward(
            r, dr=dr, dh=dh_next, b=b, w_pre=next_w_pre, w_post=w.w_post, gate=w.gate,
            alpha=self.alpha, beta=self.beta, eps=self.eps, dw_pre=dw_next, dw_post=g["w_post"],
            dgate=g["gate"])
        # each expert row's combine gate; the shared expert's rows have none
        slots = row_of.view(-1).long()
        row_gate = torch.ones(R, dtype=torch.float32, device=x.device)
        row_gate[slots] = gates.view(-1)
        dact = moe_grouped_gemm_bf16(db, w.w2, offsets, R, b_kn=True, a_row_index=token_of)
        da, drow, act = moe_swiglu_backward(a, dact, row_gate)
        moe_grouped_wgrad_bf16(db, act, offsets, R, a_row_index=token_of, out=g["w2"])
        moe_grouped_wgrad_bf16(da, h, offsets, R, b_row_index=token_of, out=g["w1"])
        drows = moe_grouped_gemm_bf16(da, w.w1, offsets, R, b_kn=True)
        # bf16, as an operand of the products below
        if balance is not None:
            _, stats, seq_offsets, token_mask, balance_alpha = balance
            dz = moe_router_backward(scores, idx, gates, drow[slots].view(T, self.k), stats.load,
                                     stats.tokens, seq_offsets, token_mask, dbalance,
                                     balance_alpha)
        else:
            picked = idx.long()
            dpicked = router_gradient(drow[slots].view(T, self.k), gates, scores.gather(1, picked))
            dz = torch.zeros_like(scores).scatter_(1, picked, dpicked).bfloat16()
        whole = torch.arange(2, dtype=torch.int32, device=x.device) * T     # one group
        moe_grouped_wgrad_bf16(dz, h, whole, T, out=g["w_router"].unsqueeze(0))
        through_router = moe_grouped_gemm_bf16(dz, w.w_router.unsqueeze(0), whole, T, b_kn=True)
        # a token's expert rows and what came through the router, summed
        dh = moe_combine(drows, torch.ones_like(gates), row_of, T * self.k,
                         residual=through_router)
        if not through_norm:
            return dx, dw_next, dh
        dx, _, _, _, _ = moe_block_norm_backward(x, dr=dx, dh=dh, w_pre=w.w_pre, eps=self.eps,
                                                 dw_pre=g["w_pre"])
        return dx, dw_next

    def clip(self, max_norm):
        """Clips self.grads in place by their global norm; returns float32
        [2] on the device: (norm, coefficient)."""
        return moe_grad_clip(self.list, max_norm)
