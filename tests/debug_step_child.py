"""Child process of test_gpu_debug_step: cases of the decode step's operators and of the weight rebuild through the
bounds-checked library, each against its 64-bit reference, the device status read after each.  Cases that give a bad
index on purpose check for its own status, over which a failed bounds check would take precedence.  Prints
"debug build ok" on success."""
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

import test_gpu_attention as attention  # noqa: E402
import test_gpu_attention_forms as forms  # noqa: E402
import test_gpu_attention_split as split  # noqa: E402
import test_gpu_decode_step as step  # noqa: E402
import test_gpu_empty_table as empty_table  # noqa: E402
import test_gpu_kv_cache as kv_cache  # noqa: E402
import test_gpu_reconstruct as rebuild  # noqa: E402
import test_gpu_sample as sample  # noqa: E402
import test_gpu_sample_masks as masks  # noqa: E402
import test_gpu_sample_paths as paths  # noqa: E402
import test_gpu_step_norm as norm  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32

CASES = [
    *[(norm.test_bf16, a) for a in ((3, 8), (3, 1032), (1, 8200), (3, 20000), (64, 512 + 8))],
    *[(norm.test_8_bits, a) for a in ((5, 1152, False), (7, 1000, True), (2, 32768, False))],
    (norm.test_bad_weight_id_flags_and_leaves_the_row, ()),
    *[(kv_cache.test_append_writes_the_defined_bytes, a) for a in (("bf16", 128, 5, 5, 48), ("e4m3", 64, 7, 1, 1024), ("e4m3", 128, 32, 8, 16))],
    *[(kv_cache.test_append_bad_index_flags_and_skips, (w,)) for w in ("page", "page_high", "seq", "position", "rope")],
    *[(kv_cache.test_read_is_exact, a) for a in (("bf16", 64, 3, 32), ("e4m3", 128, 1, 48), ("e4m3", 64, 32, 1024))],
    (kv_cache.test_read_bad_page_gives_zeros_and_flags, ()),
    (kv_cache.test_append_in_place_query_and_padding, ()),
    *[(attention.test_heads_and_lengths, (kv, dim, *heads)) for kv in ("bf16", "e4m3") for dim in (64, 128)
      for heads in ((32, 8), (12, 1), (40, 2), (1, 1))],
    *[(attention.test_pages_and_long_splits, (kv, page)) for kv in ("bf16", "e4m3") for page in (16, 48, 1024)],
    *[(attention.test_window_reads_nothing_before_it, (kv, w)) for kv in ("bf16", "e4m3") for w in (15, 100)],
    (attention.test_many_sequences, ()),
    (attention.test_bad_pages_and_lengths_flag, ()),
    *[(forms.test_short_sequences, (pages, kv, 128, *heads)) for pages in (3, 400) for kv in ("bf16", "e4m3") for heads in ((32, 8), (48, 2))],
    *[(forms.test_bad_page_and_length, (pages,)) for pages in (4, 400)],
    (split.test_a_long_sequence_among_short_ones_is_split, ("e4m3", 200, 8, 3001)),
    (empty_table.test_nothing_cached_yet, ("e4m3",)),
    *[(sample.test_vocabularies_with_mixed_settings, (d, v)) for d in (BF16, F32) for v in (1, 7, 9, 1003, 16385, 50000, 131071)],
    *[(sample.test_top_k, (d, k, p)) for d in (BF16, F32) for k in (1, 513, 5000) for p in (1.0, 0.9)],
    *[(sample.test_top_p, (d, p, t)) for d in (BF16, F32) for p in (0.1, 0.9999) for t in (0.3, 30.0)],
    *[(sample.test_masks, (d,)) for d in (BF16, F32)],
    (sample.test_odd_settings_and_noise, ()),
    (sample.test_many_rows_repeat_identically, ()),
    *[(masks.test_masks_of_several_values, (d, k)) for d in (BF16, F32) for k in masks.KINDS],
    *[(paths.test_top_p_with_noise_that_favours, (d, 40, 5003, 0.97, 8.0, "beyond")) for d in (BF16, F32)],
    *[(paths.test_unfiltered_scores_a_rounding_apart, (d, 300, 4099)) for d in (BF16, F32)],
    *[(rebuild.test_reconstruct_is_bit_exact, a) for a in ((7, 8, 0), (129, 264, 1), (513, 2048, 1))],
    (step.test_generation_matches_a_plain_forward_pass, (True,)),
]


def main():
    assert bd.bd_build_flags() & 1, "the bounds-checked library is not the one loaded"
    torch.cuda.set_device(0)
    import inspect
    for test, args in CASES:
        names = list(inspect.signature(test).parameters)
        assert len(names) == len(args), (test.__name__, names)
        test(*args)
        torch.cuda.synchronize()
        st = bd.bd_get_device_status()
        assert st == bd.BD_OK, f"{test.__name__}{args}: {bd.bd_status_string(st)}"
    print("debug build ok")


if __name__ == "__main__":
    main()
