"""The step plan and the scored calls open and close one NVTX range each, on
their early returns too (no GPU: a null pool)."""

import test_nvtx_ranges as base


def test_new_entry_points_are_nvtx_ranges(tmp_path, monkeypatch):
    monkeypatch.setattr(base, "ENTRY_CALLS", {
        "kv_plan_step": "(None, None, None, I(1), None, I(1), None, I(0), None, None, None, None, "
                        "None, None, I(0), None)",
        "paged_attention_decode_scored": "(None, None, None, None, I(1), None, I(1), I(1), F(1.0), "
                                         "I(1), None, None, S(0), None)",
        "paged_attention_prefill_scored": "(None, None, None, None, I(1), I(1), None, I(1), None, "
                                          "I(1), I(1), F(1.0), I(1), None, None)",
    })
    base.test_each_entry_point_is_one_nvtx_range(tmp_path)
