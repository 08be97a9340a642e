"""The row operators in a model: an embedding, a layer of experts behind a router, and a training step.

The operators as autograd functions (expert_dispatch, expert_combine, embedding), and a small language model that
uses all of them (RoutedModel).  Their gradients are calls of the library, which autograd does not see: they can be
taken once, and a second derivative through them is an error.  What surrounds the operators (the router's scores,
the experts' matrix products, the loss) is torch's.

    python -m sorting_lsd_radix_gb300.routed        # trains a few steps on synthetic tokens, then answers one by one
"""
from __future__ import annotations

import math
import time

import torch
from torch.autograd.function import once_differentiable

from . import gbsort


def _rows(t: torch.Tensor) -> torch.Tensor:
    """A gradient with unit stride along its rows (one that a sum sent back has stride 0)."""
    return t if t.stride(-1) == 1 or t.size(-1) == 1 else t.contiguous()


class _Dispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, expert_ids, num_experts, first_expert, row_align):
        rows, plan = gbsort.gbs_expert_dispatch(x, expert_ids, num_experts, first_expert, row_align)
        ctx.save_for_backward(plan[1])
        ctx.mark_non_differentiable(*plan)
        return rows, *plan

    @staticmethod
    @once_differentiable
    def backward(ctx, d_rows, *_):
        row_of_slot, = ctx.saved_tensors
        return gbsort.gbs_expert_combine(_rows(d_rows), row_of_slot), None, None, None, None


class _Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, rows, weights, slot_of_row, row_of_slot):
        ctx.save_for_backward(rows, weights, slot_of_row, row_of_slot)
        return gbsort.gbs_expert_combine(rows, row_of_slot, weights)

    @staticmethod
    @once_differentiable
    def backward(ctx, d_out):
        rows, weights, slot_of_row, row_of_slot = ctx.saved_tensors
        d_rows, d_weights = gbsort.gbs_expert_combine_grad(_rows(d_out), rows, slot_of_row, row_of_slot, weights)
        return d_rows, d_weights, None, None


class _Embedding(torch.autograd.Function):
    @staticmethod
    def forward(ctx, table, ids, scale, first_id, padding_id):
        ctx.save_for_backward(ids)
        ctx.vocab, ctx.dtype, ctx.args = table.shape, table.dtype, (scale, first_id, padding_id)
        return gbsort.gbs_embedding_lookup(table, ids, scale, first_id)

    @staticmethod
    @once_differentiable
    def backward(ctx, d_out):
        ids, = ctx.saved_tensors
        grad = torch.empty(ctx.vocab, dtype=ctx.dtype, device=d_out.device)
        return gbsort.gbs_embedding_grad(d_out.contiguous(), ids, grad, *ctx.args), None, None, None, None


def expert_dispatch(x, expert_ids, num_experts, first_expert=0, row_align=1):
    """(rows, slot_of_row, row_of_slot, offsets, counts) of gbs_expert_dispatch; rows carry x's gradient back."""
    return _Dispatch.apply(x, expert_ids, num_experts, first_expert, row_align)


def expert_combine(rows, weights, slot_of_row, row_of_slot):
    """gbs_expert_combine, with the gradients of the rows and of the weights (None: ones)."""
    return _Combine.apply(rows, weights, slot_of_row, row_of_slot)


def embedding(table, ids, scale=1.0, first_id=0, padding_id=None):
    """gbs_embedding_lookup, with the table's gradient; the id padding_id gets none (None or negative: no such id)."""
    return _Embedding.apply(table, ids, scale, first_id, padding_id)


class RoutedModel(torch.nn.Module):
    """Embedding, one layer of experts with a residual, and the table again as the output's matrix."""

    def __init__(self, vocab, hidden, inner, num_experts, top_k, dtype=torch.bfloat16, device="cuda"):
        super().__init__()
        self.top_k, self.scale = top_k, math.sqrt(hidden)

        def made(*shape):
            return torch.nn.Parameter(torch.randn(*shape, device=device, dtype=torch.float32).div_(
                math.sqrt(shape[-1])).to(dtype))

        self.table = made(vocab, hidden)
        self.router, self.up, self.down = made(num_experts, hidden), made(num_experts, inner, hidden), \
            made(num_experts, hidden, inner)

    def hidden(self, ids):
        x = embedding(self.table, ids, self.scale)
        score, experts = torch.topk(x.float() @ self.router.float().t(), self.top_k, dim=-1)
        rows, slot_of_row, row_of_slot, offsets, _ = expert_dispatch(x, experts, self.router.size(0))
        edge = offsets.tolist()  # the experts' products are launched by the host
        out = [torch.nn.functional.silu(rows[a:b] @ self.up[e].t()) @ self.down[e].t()
               for e, (a, b) in enumerate(zip(edge, edge[1:])) if b > a]
        y = expert_combine(torch.cat(out) if out else rows, torch.softmax(score, -1), slot_of_row, row_of_slot)
        return x + y

    def forward(self, ids):
        return self.hidden(ids).float() @ self.table.float().t()

    def loss(self, ids):
        """Each token's prediction of the next one."""
        return torch.nn.functional.cross_entropy(self(ids[:-1]), ids[1:])


def main():
    torch.manual_seed(0)
    model = RoutedModel(vocab=8192, hidden=512, inner=1024, num_experts=16, top_k=2)
    optimizer = torch.optim.AdamW(model.parameters(), lr=1e-3)
    text = (torch.arange(2049, device="cuda") * 7919) % 1021  # tokens with a rule to learn
    for step in range(20):
        started = time.perf_counter()
        optimizer.zero_grad()
        loss = model.loss(text)
        loss.backward()
        optimizer.step()
        if step % 5 == 0 or step == 19:
            print(f"step {step}: loss {loss.item():.3f}, {(time.perf_counter() - started) * 1e3:.1f} ms")
    with torch.no_grad():
        token, answer = text[:1], []
        for _ in range(8):
            token = model(token).argmax(-1)
            answer.append(int(token))
    print("answer", answer, "text", text[1:9].tolist())


if __name__ == "__main__":
    main()
