"""Rounds of speculative decoding around one attention layer, on a GPU.

A toy target (one attention layer, a projection to the vocabulary) runs gamma + 1 new tokens
of every sequence over its paged cache, its logits get penalties and a mask, a drafter that
knows the target's logits up to noise proposes the next tokens, and spec_verify decides.
Rejected tokens need no clean-up: the cache lengths advance by what was accepted, and the
next round writes over the rest.

    python examples/target_round.py [--batch 32] [--gamma 7] [--prompt 2000] [--rounds 20]

Random weights; what it prints is the mean number of accepted tokens, the time of a round and
whether any sequence reported a problem.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import speculative_decoding_verification_20_gb300 as sv  # noqa: E402


class Target:
    def __init__(self, vocab, q_heads, kv_heads, dim, batch, context, page_size, device):
        g = torch.Generator(device).manual_seed(0)
        rnd = lambda *s: torch.randn(s, generator=g, device=device, dtype=torch.float32)
        self.Hq, self.Hkv, self.D, self.vocab = q_heads, kv_heads, dim, vocab
        width = q_heads * dim
        self.embed = rnd(vocab, width).bfloat16()
        self.qkv = (rnd(width, (q_heads + 2 * kv_heads) * dim) / width ** 0.5).bfloat16()
        self.head = (rnd(width, vocab) * 3.0 / width ** 0.5).bfloat16()
        per_seq = (context + page_size - 1) // page_size
        self.cache = sv.PagedCache(batch * per_seq, page_size, kv_heads, dim, device=device)
        self.page_table = torch.randperm(batch * per_seq, generator=g, device=device).to(torch.int32).view(batch, per_seq)
        self.table = sv.rotary_table(per_seq * page_size, dim, device=device)

    def __call__(self, tokens, lens, max_context, status):
        """Logits [B, N, vocab] of tokens [B, N] appended at positions lens[b] and on."""
        B, N = tokens.shape
        x = self.embed[tokens.long()]
        qkv = (x @ self.qkv).view(B, N, self.Hq + 2 * self.Hkv, self.D)
        q, k, v = qkv.split([self.Hq, self.Hkv, self.Hkv], dim=2)
        q = sv.rotate_append(q, k, v, self.table, self.cache, self.page_table, lens, row_status=status)
        o = sv.paged_attention(q, self.cache, self.page_table, lens, max_context=max_context, row_status=status)
        return (x + o.reshape(B, N, -1)) @ self.head


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--batch", type=int, default=32)
    ap.add_argument("--gamma", type=int, default=7)
    ap.add_argument("--prompt", type=int, default=2000)
    ap.add_argument("--rounds", type=int, default=20)
    ap.add_argument("--vocab", type=int, default=32000)
    a = ap.parse_args()
    dev = torch.device("cuda:0")
    B, G, V = a.batch, a.gamma, a.vocab
    context = a.prompt + (a.rounds + 1) * (G + 1)
    target = Target(V, 32, 8, 128, B, context, 64, dev)
    status = torch.zeros(B, dtype=torch.int32, device=dev)
    g = torch.Generator(dev).manual_seed(1)
    prompt = torch.randint(0, V, (B, a.prompt), generator=g, device=dev, dtype=torch.int32)
    lens = torch.zeros(B, dtype=torch.int32, device=dev)
    history = sv.TokenHistory(B, V, device=dev)
    history.load(prompt, torch.full((B,), a.prompt))
    # the prompt in chunks; the last token starts the first round
    at = 0
    while at < a.prompt - 1:
        n = min(2048, a.prompt - 1 - at)
        target(prompt[:, at:at + n], lens, context, status)
        at += n
        lens += n
    last = prompt[:, -1:]
    banned = torch.zeros((B, (V + 31) // 32), dtype=torch.int32, device=dev)
    banned[:, 0] = 1  # token 0 is never allowed
    accepted, times = [], []
    for step in range(a.rounds):
        begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        begin.record()
        # the drafter: the target's own next-token logits with noise, token by token
        draft, tok = [], last
        q_rows = []
        for i in range(G):
            rows = target(tok, lens + i, context, status)
            rows = sv.process_logits(rows + 0.3 * torch.randn(rows.shape, generator=g, device=dev, dtype=rows.dtype),
                                     history=history, repetition=1.1, mask=~banned)
            tok = rows[:, 0].float().softmax(-1).multinomial(1, generator=g).to(torch.int32)
            q_rows.append(rows)
            draft.append(tok)
        x = torch.cat(draft, 1)
        logits = target(torch.cat((last, x), 1), lens, context, status)
        p_rows = sv.process_logits(logits, history=history, draft_tokens=x, repetition=1.1, mask=~banned)
        res = sv.spec_verify(p_rows, torch.cat(q_rows, 1), x, 1.0, seed=step)
        history.add(res["out_tokens"])
        n = res["accepted_len"]
        last = res["out_tokens"].gather(1, n.long()[:, None])
        lens = lens + n + 1
        status |= res["row_status"]
        end.record()
        accepted.append(n)
        times.append((begin, end))
    torch.cuda.synchronize()
    ms = sorted(b.elapsed_time(e) for b, e in times)[len(times) // 2]
    print(f"accepted {torch.stack(accepted).float().mean().item():.2f} of {G} drafts a round, {ms:.2f} ms a round, "
          f"sequences with a problem: {int((status != 0).sum())}")


if __name__ == "__main__":
    main()
