"""Child process of test_gpu_debug_long: cases of the long-context operators through the bounds-checked library, each against its
64-bit reference, the device status read after each.  Prints "debug build ok" on success."""
import os
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
for p in (ROOT, HERE):
    if p not in sys.path:
        sys.path.insert(0, p)

import torch  # noqa: E402

from bit_delta_tenant_gb300 import bitdelta as bd  # noqa: E402

bd.load_library(bd.LIB_DEBUG_PATH)

import test_gpu_decode_step_long as step  # noqa: E402
import test_gpu_four_bits as four  # noqa: E402
import test_gpu_prompt as prompt  # noqa: E402
import test_gpu_prompt_calls as calls  # noqa: E402
import test_gpu_rotary as rotary  # noqa: E402

KINDS = prompt.KINDS
CASES = [
    *[(prompt.test_heads_and_lengths, (kv, dim, *heads)) for kv in KINDS for dim in (64, 128) for heads in ((32, 8), (48, 2), (150, 1), (1, 1))],
    *[(prompt.test_pages_and_long_prompts, (kv, page)) for kv in KINDS for page in (16, 48, 1024)],
    *[(prompt.test_few_queries_over_many_keys, (kv, [40, 1], [3000, 5000])) for kv in KINDS],
    *[(prompt.test_rules, (kv, kw)) for kv in KINDS for kw in prompt.RULES],
    *[(prompt.test_unseen_infinities_and_nan, (kv, 128)) for kv in KINDS],
    *[(calls.test_bad_pages_hide_their_keys, (kv, 16)) for kv in KINDS],
    (calls.test_many_sequences, ("e2m1",)),
    (calls.test_bad_lengths_and_offsets_flag, ()),
    *[(four.test_heads_and_lengths, (dim, *heads)) for dim in (64, 128) for heads in ((32, 8), (12, 1), (48, 2))],
    *[(four.test_rules, (kv, lengths, dict(cap=5.0, slopes=True, first=True, window=100), 128, (32, 2))) for kv in KINDS
      for lengths in ([4099, 1, 1000, 0, 2500], [70, 500, 0, 3, 512, 128])],
    (four.test_bytes_of_every_size, (128,)),
    *[(four.test_read_is_exact, a) for a in ((64, 3, 32), (128, 1, 48))],
    *[(rotary.test_table, (n, dim, dict())) for n, dim in ((1, 2), (4097, 128), (5, 10))],
    *[(rotary.test_parts_and_layouts, (kv, i, 128, 80, 1, 40)) for kv in KINDS for i in (False, True)],
    (step.test_generation_matches_a_plain_forward_pass, (True,)),
]


def main():
    assert bd.bd_build_flags() & 1, "the bounds-checked library is not the one loaded"
    torch.cuda.set_device(0)
    for test, args in CASES:
        test(*args)
        torch.cuda.synchronize()
        st = bd.bd_get_device_status()
        assert st == bd.BD_OK or test is calls.test_bad_pages_hide_their_keys and st == bd.BD_ERR_BAD_INDEX, f"{test.__name__}{args}: {bd.bd_status_string(st)}"
    print("debug build ok")


if __name__ == "__main__":
    main()
