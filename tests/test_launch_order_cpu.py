"""Every kernel that may start beside the end of the stream's kernel before it
waits for that kernel (checked in the sources, without a GPU)."""
import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "chunk_scheduled_communication_gb300", "csrc")


def closing(text, at, pair):
    """Index of the bracket that closes the one at `at`."""
    depth = 0
    for i in range(at, len(text)):
        depth += (text[i] == pair[0]) - (text[i] == pair[1])
        if depth == 0:
            return i
    raise AssertionError("unbalanced source")


def sources():
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))):
        yield re.sub(r"//[^\n]*|/\*.*?\*/", "", open(path).read(), flags=re.S)


def early_kernels():
    names = set()
    for text in sources():
        for m in re.finditer(r"(?<!\w)launch_early\(", text):
            call = text[m.start():closing(text, m.end() - 1, "()")]
            if "cudaError_t launch_early" not in text[max(m.start() - 12, 0):m.end()]:
                names |= set(re.findall(r"\b(\w+_kernel)\b", call))
    return names


def body(name):
    found = []
    for text in sources():
        for m in re.finditer(r"__global__[^;{]*?\b" + name + r"\(", text):
            begin = text.index("{", closing(text, m.end() - 1, "()"))
            found.append(text[begin:closing(text, begin, "{}")])
    assert len(found) == 1, (name, len(found))
    return found[0]


def test_every_early_kernel_waits_in_every_thread():
    names = early_kernels()
    assert {"rope_kernel", "norm_grad_kernel", "window_fwd_kernel", "window_decode_kernel"} <= names
    for name in sorted(names):
        text = body(name)
        assert text.count("ptx::grid_wait();") == 1, name
        before = re.sub(r"\[&\]\([^)]*\)\s*\{[^{}]*\}", "", text[:text.index("ptx::grid_wait();")])  # without lambdas
        # unconditional: no block is open at the wait, nothing returns before it
        assert before.count("{") - before.count("}") == 1, name
        assert not re.search(r"\breturn\b", before), name


def test_kernel_attributes_are_set_by_plans_alone():
    """A kernel's attributes are the context's: a call that set them would change
    them under another host thread's launch."""
    seen = 0
    for text in sources():
        if "launch_early(" not in text:
            continue
        for m in re.finditer(r"cudaFuncSetAttribute\(", text):
            # the function that the call stands in: the last one at file level before it
            name = re.findall(r"^(?:template <[^>]*> )?[\w:]+ (\w+)\([^;]*?\) \{", text[:m.start()], flags=re.M)[-1]
            assert name.endswith("prepare"), name
            seen += 1
    assert seen >= 5


def test_a_plan_is_on_the_device_when_it_is_made():
    """What a plan's creation copies and clears has reached the device before the
    plan is handed out: a stream of the caller's need not wait for the default one."""
    made = 0
    for text in sources():
        for m in re.finditer(r"^int syn_(rope|window|decode)_plan_create\(", text, flags=re.M):
            begin = text.index("{", closing(text, m.end() - 1, "()"))
            create = text[begin:closing(text, begin, "{}")]
            # (the null pointer at the start aside)
            last = create.rindex("*out = pl;")
            assert "cudaDeviceSynchronize()" in create[:last], m.group(1)
            made += 1
    assert made == 3


def test_a_cleared_error_word_is_cleared_before_the_next_call():
    found = 0
    for text in sources():
        for m in re.finditer(r"^int syn_\w*sync_status\(", text, flags=re.M):
            begin = text.index("{", closing(text, m.end() - 1, "()"))
            clear = text[begin:closing(text, begin, "{}")]
            assert "cudaDeviceSynchronize()" in clear[clear.rindex("cudaMemset("):], m.group(0)
            found += 1
    assert found >= 4


def test_decode_waits_leave_a_warp_whole_and_a_lost_copy_ends_the_loading():
    text = next(t for t in sources() if "window_decode_kernel(" in t and "__global__" in t)
    at = text.index("auto landed")
    wait = text[at:closing(text, text.index("{", at), "{}")]
    # the matrix loads and products behind it need converged warps
    assert wait.count("return") == 1 and "__syncwarp();" in wait[:wait.index("return")]
    # reported at the limit, then waited for again, with a limit of its own
    assert wait.index("SYN_ERR_TIMEOUT") < wait.index("limit += kDrainNs")
    # a barrier whose rows never came is not armed again
    assert "&& !lost) load(t +" in text and "if (!lost) lost = !landed(" in text
    assert "SYN_ERR_TIMEOUT ?" in text


def test_producers_stop_after_a_wait_that_ran_out():
    """A barrier whose copies are still under way is not armed again: between a
    producer's wait for a free stage and its next copies it asks whether a wait ran
    out, and the waits on the way out have a limit of their own."""
    found = 0
    for text in sources():
        at = text.find("if (warp == 0) {")
        if "tma_load_3d" not in text or "__global__" not in text:
            continue
        producer = text[at:closing(text, text.index("{", at), "{}")]
        waits = [m.start() for m in re.finditer(r"(?<!\w)wait_bar\(", producer)]
        armed = [m.start() for m in re.finditer("mbar_arrive_expect_tx", producer)]
        assert len(waits) == len(armed) > 0
        for w, a in zip(waits, armed):
            assert w < producer.index("aborted(abort)", w) < a
        found += 1
    assert found == 3
    shared = next(t for t in sources() if "void drain_bar" in t and "launch_early" in t)
    wait = shared[shared.index("void wait_long"):shared.index("void wait_bar")]
    assert "kDrainNs" in wait
