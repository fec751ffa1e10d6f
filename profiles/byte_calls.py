"""Three calls of one operator of the cache held in 8 bits, for a profiler: python profiles/byte_calls.py CASE (see CASES)."""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bit_kv_cache_ott_gb300 as ott  # noqa: E402

#        B  Hq  Hkv d    G    T     n  topk
CASES = {
    "store": (4, 32, 32, 128, 64, 4096, 0, 0),      # k_byte_append, k_byte_read
    "decode": (16, 32, 32, 128, 64, 4096, 0, 0),    # k_byte_rows, k_byte_combine
    "long": (1, 32, 8, 128, 64, 131071, 0, 0),      # the same, few units
    "rows16": (8, 32, 8, 128, 64, 8192, 4, 0),      # k_byte_rows with 16 columns
    "tiles": (1, 32, 8, 128, 64, 16384, 2048, 0),   # k_byte_tiles, k_byte_tiles_combine
    "sparse": (1, 32, 8, 128, 64, 131071, 0, 256),  # k_byte_select, k_byte_rows
}


def main(case):
    B, Hq, Hkv, d, G, T, n, topk = CASES[case]
    new = lambda h, x: torch.randn(B, h, x, d, device="cuda").half()
    c = ott.ByteCache(B, Hq, Hkv, d, G, max_tokens=T)
    K, V = new(Hkv, T), new(Hkv, T)
    q, k, v = new(Hq, max(n, 1)), new(Hkv, max(n, 1)), new(Hkv, max(n, 1))
    c.prefill(K, V)
    torch.cuda.synchronize()
    for _ in range(3):
        if case == "store":
            c.reset()
            c.append_chunk(K, V)
            c.read(0, T, K, V)
        elif n:
            c.chunk_attn(q, k, v)
        else:
            c.decode_attn_topk(q[:, :, 0].contiguous(), topk)
    torch.cuda.synchronize()
    c.check_device()


if __name__ == "__main__":
    for name in sys.argv[1:]:
        main(name)
