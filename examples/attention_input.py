"""The input side of an attention block on an int8 layer, prompt and decode.

    python examples/attention_input.py [--tokens 1000] [--steps 4]

One fused projection with int8 weights gives a row of queries, keys and values
per token; queries and keys are normed per head and rotated in place; keys and
values go to the slots of a paged cache.  The same steps serve a prompt and
single tokens: the script runs a batch of prompts, decodes a few tokens, and
checks that the cache then holds, bit for bit, what one pass over the longer
sequences writes.
"""

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import blockwise_bit_codebook_amd as kb  # noqa: E402


class AttentionInput:
    """Weights, rotation table and cache of one block."""

    def __init__(self, hidden, heads, kv_heads, dim, max_pos, pages, page_size, device="cuda", seed=0):
        g = torch.Generator(device).manual_seed(seed)
        self.heads, self.kv_heads, self.dim, self.page_size = heads, kv_heads, dim, page_size
        width = (heads + 2 * kv_heads) * dim
        w = torch.randn(width, hidden, device=device, generator=g) * hidden ** -0.5
        self.w_codes, self.w_scale = kb.quantize_rows_int8(w.bfloat16())
        self.q_weight = torch.ones(dim, device=device, dtype=torch.bfloat16)
        self.k_weight = torch.ones(dim, device=device, dtype=torch.bfloat16)
        # a context four times longer than the one of max_pos / 4 trained on
        freq, amplitude = kb.rope_frequencies(dim, scaling="yarn", factor=4.0, original_length=max_pos // 4)
        self.table = kb.rope_table(freq, max_pos, amplitude=amplitude, device=device)
        self.k_cache, self.v_cache = (
            torch.zeros(pages, page_size, kv_heads, dim, device=device, dtype=torch.bfloat16) for _ in range(2))

    def __call__(self, x, positions, slots):
        """x [tokens, hidden] -> rotated queries [tokens, heads, dim]; keys and values go to the cache."""
        qkv = kb.linear_int8_dynamic(x, self.w_codes, self.w_scale)
        tokens, h, k = x.shape[0], self.heads * self.dim, self.kv_heads * self.dim
        queries = qkv[:, :h].view(tokens, self.heads, self.dim)
        keys = qkv[:, h:h + k].view(tokens, self.kv_heads, self.dim)
        values = qkv[:, h + k:].view(tokens, self.kv_heads, self.dim)
        kb.qk_norm_rope(queries, keys, self.q_weight, self.k_weight, positions, self.table, q_out=queries, k_out=keys)
        kb.append_kv_paged(keys, values, slots, self.k_cache, self.v_cache)
        return queries


def _slots(pages_of, positions, sequence, page_size):
    """Slot of each token: its sequence's page for the position, and the place in it."""
    return pages_of[sequence, positions // page_size] * page_size + positions % page_size


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=1000, help="tokens of the prompts together")
    ap.add_argument("--steps", type=int, default=4, help="tokens decoded for each sequence")
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--heads", type=int, default=32)
    ap.add_argument("--kv-heads", type=int, default=8)
    ap.add_argument("--dim", type=int, default=128)
    a = ap.parse_args(argv)
    dev = "cuda"
    lengths = [a.tokens // 2, a.tokens // 3, a.tokens - a.tokens // 2 - a.tokens // 3]
    page_size, per = 16, -(-(max(lengths) + a.steps) // 16)
    pages = len(lengths) * per
    pages_of = torch.randperm(pages, device=dev).view(len(lengths), per)

    def tokens_of(first, last):
        """Positions and sequences of tokens first[i] .. last[i] - 1 of every sequence."""
        pos = torch.cat([torch.arange(f, n, device=dev) for f, n in zip(first, last)])
        seq = torch.cat([torch.full((n - f,), i, device=dev) for i, (f, n) in enumerate(zip(first, last))])
        return pos, seq

    ends = [n + a.steps for n in lengths]
    x = [torch.randn(n, a.hidden, device=dev).bfloat16() for n in ends]
    make = lambda: AttentionInput(a.hidden, a.heads, a.kv_heads, a.dim, 4096, pages, page_size)  # noqa: E731

    # the prompts, then single tokens
    block = make()
    pos, seq = tokens_of([0] * len(lengths), lengths)
    last = block(torch.cat([t[:n] for t, n in zip(x, lengths)]), pos, _slots(pages_of, pos, seq, page_size))
    torch.cuda.synchronize()
    start = time.perf_counter()
    for s in range(a.steps):
        pos, seq = tokens_of([n + s for n in lengths], [n + s + 1 for n in lengths])
        last = block(torch.stack([t[n + s] for t, n in zip(x, lengths)]), pos, _slots(pages_of, pos, seq, page_size))
    torch.cuda.synchronize()
    decode_us = (time.perf_counter() - start) / a.steps * 1e6

    # the same tokens in one pass
    whole = make()
    pos, seq = tokens_of([0] * len(lengths), ends)
    queries = whole(torch.cat(x), pos, _slots(pages_of, pos, seq, page_size))
    ends_at = torch.tensor(ends, device=dev).cumsum(0) - 1
    same = (torch.equal(block.k_cache, whole.k_cache) and torch.equal(block.v_cache, whole.v_cache)
            and torch.equal(last, queries[ends_at]))
    print(f"prompts of {lengths} tokens and {a.steps} steps of {len(lengths)}: "
          f"{'the same bits as in one pass' if same else 'DIFFERENT from one pass'}; {decode_us:.0f} us a step "
          f"with the slots' arithmetic")
    if not same:
        raise SystemExit(1)


if __name__ == "__main__":
    main()
