"""Three calls of one chunk operator, for a profiler: python profiles/chunk_calls.py CASE (see CASES)."""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bit_kv_cache_ott_gb300 as ott  # noqa: E402

#        B  Hq  Hkv d    T      n (per sequence, or a list)  window sinks
CASES = {
    "long": (1, 32, 8, 128, 16384, 2048, 0, 0),                       # k_chunk_tiles, tiles cut between CTAs
    "mixed": (8, 32, 32, 128, 4096, [257, 0, 96, 1, 200, 33, 64, 128], 0, 0),
    "short": (1, 32, 8, 128, 0, 1024, 0, 0),                          # causal over the chunk alone
    "rows4": (32, 32, 32, 128, 4096, 4, 0, 0),                        # rows mode of k_decode
    "rows8": (32, 32, 32, 128, 4096, 8, 0, 0),                        # k_chunk_rows<128, 1>
    "rows16": (32, 32, 32, 128, 4096, 16, 0, 0),                      # k_chunk_rows<128, 2>
    "window": (32, 32, 32, 128, 4096, 0, 1024, 4),                    # a windowed step
    "append": (1, 32, 8, 128, 0, 1024, 0, 0),                         # three appends of a chunk
}


def main(case):
    B, Hq, Hkv, d, T, n, window, sinks = CASES[case]
    lens = n if isinstance(n, list) else None
    m = max(n) if lens else max(n, 1)
    new = lambda h, x: torch.randn(B, h, x, d, device="cuda").half()
    c = ott.OTTCache(B, Hq, Hkv, d, 128, 32, 32, max_tokens=T + 3 * m, ragged=lens is not None)
    if T:
        c.prefill(new(Hkv, T), new(Hkv, T))
    q, k, v = new(Hq, m), new(Hkv, m), new(Hkv, m)
    torch.cuda.synchronize()
    for _ in range(3):
        if case == "append":
            c.append_chunk(k, v)
        elif case == "window":
            c.decode_attn_window(q[:, :, 0].contiguous(), window, sinks)
        else:
            c.chunk_attn(q, k, v, lens=lens)
    torch.cuda.synchronize()
    c.check_device()


if __name__ == "__main__":
    main(sys.argv[1])
