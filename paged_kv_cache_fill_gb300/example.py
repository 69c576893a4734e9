"""A first call sequence through the Python binding (needs a GB300):
slot filling, a BF16 cache write, a paged decode with split-KV and a chunked
prefill over the same cache; then an FP8 cache with a scale for each block and
head, a fork of one of its sequences, and a decode of all three under a window
with sinks. PyTorch supplies the device memory; every array
is a contiguous CUDA tensor and every size is passed explicitly.

Run: python -m paged_kv_cache_fill_gb300.example
"""
import torch

import paged_kv_cache_fill_gb300 as pk


def main() -> None:
    dev, H, Hq, D, bs, nb, mbps = "cuda", 8, 32, 128, 16, 1024, 64
    seq_lens = torch.tensor([37, 100], dtype=torch.int32, device=dev)
    block_tables = torch.randperm(nb, device=dev)[:2 * mbps].view(2, mbps).to(torch.int32)
    k_cache = torch.empty((nb, bs, H, D), dtype=torch.bfloat16, device=dev)
    v_cache = torch.empty_like(k_cache)

    # write every position's K and V through its slot
    n = int(seq_lens.sum())
    slots = torch.empty(n, dtype=torch.int64, device=dev)
    off = 0
    for s, L in enumerate(seq_lens.tolist()):
        pk.kv_fill_slots(slots[off:off + L], block_tables[s], 0, L, bs)
        off += L
    key = torch.randn(n, H * D, device=dev).to(torch.bfloat16)
    value = torch.randn(n, H * D, device=dev).to(torch.bfloat16)
    pk.kv_write_bf16(key, value, k_cache, v_cache, slots, n, H, D, bs, H * D, H * D)

    # decode one query token per sequence (a registered workspace enables split-KV)
    pk.kv_set_decode_workspace(torch.empty(pk.kv_decode_workspace_bytes(mbps, 2, Hq, H, D, bs),
                                           dtype=torch.uint8, device=dev))
    q = torch.randn(2, Hq * D, device=dev).to(torch.bfloat16)
    out = torch.empty(2, Hq, D, device=dev)
    pk.paged_decode_attn_bf16(q, k_cache, v_cache, out, block_tables, seq_lens, mbps, 2, Hq, H, D, bs,
                              D ** -0.5, Hq * D, 0)

    # or attend the last 5 and 20 positions as a causal chunk of query tokens
    qsl = torch.tensor([0, 5, 25], dtype=torch.int32, device=dev)
    qp = torch.randn(25, Hq * D, device=dev).to(torch.bfloat16)
    outp = torch.empty(25, Hq, D, device=dev)
    pk.paged_prefill_attn_bf16(qp, k_cache, v_cache, outp, block_tables, seq_lens, qsl, mbps, 2, 25, Hq, H, D,
                               bs, D ** -0.5, Hq * D, 0)

    # the same tokens in an FP8 cache with a scale per (block, KV head), in three
    # table rows of which the third is still free
    tables3 = torch.full((3, mbps), -1, dtype=torch.int32, device=dev)
    tables3[:2] = torch.where(torch.arange(mbps, device=dev) * bs < seq_lens[:, None], block_tables, -1)
    lens3 = torch.tensor([37, 100, 0], dtype=torch.int32, device=dev)
    ref_counts = torch.zeros(nb, dtype=torch.int32, device=dev)
    ref_counts[tables3[tables3 >= 0].long()] = 1
    kq = torch.empty((nb, bs, H, D), dtype=torch.uint8, device=dev)
    vq = torch.empty_like(kq)
    k_scales = torch.empty((nb, H), device=dev)
    v_scales = torch.empty_like(k_scales)
    new = torch.tensor([0, 37, 137, 137], dtype=torch.int32, device=dev)
    pk.kv_write_fp8_block(key, value, kq, vq, k_scales, v_scales, tables3, lens3, new, mbps, 3, n, H, D, bs, H * D,
                          H * D)

    # row 2 becomes a fork of row 1: full blocks shared, the partial one copied
    src = torch.tensor([1], dtype=torch.int32, device=dev)
    dst = torch.tensor([2], dtype=torch.int32, device=dev)
    copy_src, copy_dst = torch.empty_like(src), torch.empty_like(src)
    pk.kv_fork_blocks(tables3, lens3, ref_counts, src, dst, copy_src, copy_dst, 1, mbps, 3, nb, bs)
    pk.kv_copy_blocks([kq, vq, k_scales, v_scales], copy_src, copy_dst, 1, nb)

    # decode under a window of 64 positions and 4 sinks
    q3 = torch.randn(3, Hq * D, device=dev).to(torch.bfloat16)
    out3 = torch.empty(3, Hq, D, device=dev)
    pk.paged_decode_attn_fp8_block(q3, kq, vq, k_scales, v_scales, out3, tables3, lens3, mbps, 3, Hq, H, D, bs,
                                   D ** -0.5, Hq * D, 64, 4)
    assert pk.kv_get_device_error() == 0   # synchronises; nonzero bits name a fault
    pk.kv_set_decode_workspace(None)
    print("decode output", tuple(out.shape), "prefill output", tuple(outp.shape), "FP8 decode of the fork",
          tuple(out3.shape))


if __name__ == "__main__":
    main()
