"""Decoding over an 8-bit KV page cache whose 16-bit pages rest, losslessly
compressed, in pinned host memory.

The prompt's keys and values are compressed once, a page of 16 tokens of one
head to a row (ibp_compress), the archive.  The GPU restores them from there
(ibp_gather_decompress), appends them to 8-bit pages (ibp_kv_append) and
decodes: each step appends a token, attends over the pages and counts the
attention weight that every page receives (ibp_kv_attention).  Whenever a
sequence has outgrown its budget, each head gives up its lightest pages
(ibp_kv_evict), whose places take the tokens that come.  At the end the pages
that were given up are fetched back from the archive, bit for bit.

    python examples/kv_decode.py [--seqs 4] [--heads 8] [--prompt 2048] [--steps 64]
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

from lossless_bit_level_amd import ibp, ibp_kv  # noqa: E402

PAGE = 16  # tokens


def random_kv(gen, *shape):
    """bfloat16 N(0, 1) with four wide channels."""
    x = torch.randn(shape, generator=gen, device="cuda")
    x[..., :4] *= 20.0
    return x.to(torch.bfloat16)


def archive(x):
    """[seqs, tokens, heads, d] as compressed pages (seq, head, 16 tokens) in
    pinned host memory: metadata, slots, flags."""
    seqs, tokens, heads, d = x.shape
    rows = x.permute(0, 2, 1, 3).reshape(seqs * heads * (tokens // PAGE), PAGE * d).contiguous()
    rows = rows.view(torch.uint8)
    md, _ = ibp.ibp_build_metadata(rows[:4096])
    slots = torch.empty(rows.shape, dtype=torch.uint8, pin_memory=True)
    slots, flags, row_bits = ibp.ibp_compress(md, rows, slots=slots)
    torch.cuda.synchronize()
    stored = int((row_bits.long() + 31).div(32, rounding_mode="floor").mul(4).clamp(max=rows.shape[1]).sum())
    return (md, slots, flags), stored / rows.numel()


def restore(arch, ids, d):
    """Pages `ids` of an archive, [len(ids), 16, d] bfloat16."""
    return ibp.ibp_gather_decompress(*arch, ids).view(torch.bfloat16).reshape(-1, PAGE, d)


def main(seqs=4, heads=8, group=4, d=128, prompt=2048, steps=64, keep=96, seed=0, quiet=False):
    dev = torch.device("cuda")
    gen = torch.Generator(dev).manual_seed(seed)
    k, v = random_kv(gen, seqs, prompt, heads, d), random_kv(gen, seqs, prompt, heads, d)
    (k_arch, k_ratio), (v_arch, v_ratio) = archive(k), archive(v)
    per_head = prompt // PAGE

    # a pool with room for the prompt and the steps of every head
    m = per_head + -(-steps // PAGE) + 1
    n_pages = seqs * heads * m
    codes = [torch.zeros(n_pages, PAGE * d, dtype=torch.uint8, device=dev) for _ in range(2)]
    scales = [torch.ones(n_pages, device=dev) for _ in range(2)]
    cache = ibp_kv.ibp_kv_cache(codes[0], scales[0], codes[1], scales[1], PAGE, d)
    pages = torch.randperm(n_pages, generator=gen, device=dev).to(torch.int32).reshape(seqs, heads, m)
    weights = torch.zeros(seqs, heads, m, device=dev)
    lengths = torch.full((seqs, heads), prompt, dtype=torch.int32, device=dev)

    # which archive row a pool page holds, -1 for tokens of the answer, and which
    # rows have been given up (the last entry is no row's)
    rows = torch.arange(seqs * heads * per_head, device=dev).reshape(seqs, heads, per_head)
    source = torch.full((n_pages,), -1, dtype=torch.int64, device=dev)
    source[pages[..., :per_head].long()] = rows
    given_up = torch.zeros(rows.numel() + 1, dtype=torch.bool, device=dev)
    place = torch.arange(m, device=dev)

    def held(lengths):
        """Places of the table that hold tokens, [seqs, heads, m]."""
        return place < -(-lengths // PAGE)[..., None]

    # the prompt: archive -> 16-bit pages -> 8-bit pages
    shape = (seqs, heads, prompt, d)
    from_archive = [restore(a, rows.reshape(-1), d).reshape(shape).transpose(1, 2) for a in (k_arch, v_arch)]
    ibp_kv.ibp_kv_append(cache, pages, lengths, *from_archive)

    evicted = 0
    for _ in range(steps):
        q = torch.randn(seqs, 1, heads * group, d, generator=gen, device=dev).to(torch.bfloat16)
        lengths += 1
        begun = pages.gather(2, ((lengths - 1) // PAGE)[..., None].long())[..., 0].long()
        source[begun] = torch.where((lengths - 1) % PAGE == 0, -1, source[begun])  # a page filled anew
        ibp_kv.ibp_kv_append(cache, pages, lengths, random_kv(gen, seqs, 1, heads, d),
                             random_kv(gen, seqs, 1, heads, d))
        out, weights = ibp_kv.ibp_kv_attention(cache, pages, lengths, q, weights=weights,
                                               weights_out=weights)
        before = lengths
        pages, weights, lengths = ibp_kv.ibp_kv_evict(pages, weights, lengths, PAGE, keep_pages=keep,
                                                      sink_pages=1, recent_pages=4)
        evicted += (before - lengths).sum() // PAGE
        given_up[torch.where(held(before) & ~held(lengths), source[pages.long()], -1)] = True

    # what the heads gave up, from the archive: the original bits.  With what they
    # still hold these are the prompt's pages, each once.
    gone = given_up[:-1].nonzero()[:, 0]
    kept = source[pages.long()][held(lengths)]
    assert torch.equal(torch.cat([gone, kept[kept >= 0]]).sort()[0], rows.reshape(-1))
    for x, a in ((k, k_arch), (v, v_arch)):
        want = x.transpose(1, 2).reshape(-1, PAGE, d)[gone]
        assert torch.equal(restore(a, gone, d).view(torch.int16), want.view(torch.int16))
    if not quiet:
        print(f"archive: {k_ratio:.3f} (keys) and {v_ratio:.3f} (values) of the 16-bit pages, in host memory")
        print(f"{steps} steps of {seqs} sequences: {int(evicted)} pages given up, "
              f"{int(lengths.sum())} tokens held in {seqs * heads} heads, "
              f"{len(gone)} pages of the prompt fetched back bit for bit")
    return out, lengths, weights


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, default in (("seqs", 4), ("heads", 8), ("group", 4), ("prompt", 2048), ("steps", 64), ("keep", 96)):
        ap.add_argument(f"--{name}", type=int, default=default)
    main(**vars(ap.parse_args()))
