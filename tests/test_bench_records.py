"""The counter record that the benchmark reports HBM bytes from belongs to the
kernel sources of this tree: bench.py leaves the bytes out otherwise."""


def test_traffic_record_is_of_these_sources():
    import bench
    rec = bench.load_traffic()
    assert rec is not None, "profiles/traffic_chunk_fwd_layer_8x4096x16_d128.json was taken on other kernel sources"
    assert rec["source_hash"] == bench.kernel_source_hash()
